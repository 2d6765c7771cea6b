// gdn_moe.cu -- the mixture-of-experts feed-forward ("qwen35moe -- Forward-Pass
// Design (Pantheon port)", the MoE section): with the chosen experts e and weights
// w of each token x (gdn_route.cu),
//   out = residual + sum_e w_e down_e (silu(gate_e x) * (up_e x))
//         + sigmoid(x . sh_router) sh_down (silu(sh_gate x) * (sh_up x)).
//
// Bound by the weights: even a long prompt has only a hundred tokens per expert. So the
// weights are the tensor core's A operand (128 rows of a weight per product) and an
// expert's tokens its N (16 to 128), each weight tile passing through shared
// memory once per 128 tokens.
//  - The pairs (token, expert) enter their expert's list as they are routed (or by
//    moe_place, for a given routing).
//  - moe_experts: one persistent kernel for both halves. Units of work are handed out
//    in order by a counter: first (expert, 128 rows of gate and of up, token
//    tile), whose epilogue writes h = silu(g) * u; then (expert, 256 rows of down,
//    token tile), which wait until their tile's h is complete. A unit waits only for units
//    that were handed out before it, so it never waits for a CTA that is not running.
//    Both kinds are the same pipeline: two A tiles and one B tile per stage of
//    64 along K, two accumulators, double-buffered against the epilogue. Token rows
//    come by TMA gathers of four rows (tiles of 32 tokens) or by asynchronous copies (of 128).
//    256 tokens: 227 us, HBM at 6.9 TB/s. 4,096 tokens: 326 us, 1.85 GB of HBM traffic and
//    12.4 TB/s from L2 into the SMs.
//  - moe_combine: residual, the pairs' outputs in slot order, the shared expert with its gate.
#include <mutex>

#include "gdn_moe.cuh"
#include "gdn_tc.cuh"
#include "gdn_tma.cuh"

namespace gdn {

__device__ unsigned int g_moe_error;      // GDN_ERR_TIMEOUT if a bounded wait gave up

// ------------------------------------------------------------------ places

__global__ void __launch_bounds__(256) moe_zero_kernel(int *state, int n)
{
    grid_dep_wait();
    grid_dep_launch();
    for (int i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256) state[i] = 0;
}

// Places of a given routing.
__global__ void __launch_bounds__(256) moe_place_kernel(const int32_t *ids, int pairs, int k, int E, MoePlaces places)
{
    grid_dep_wait();
    grid_dep_launch();
    const int p = blockIdx.x * 256 + threadIdx.x;
    if (p >= pairs) return;
    const int e = ids[p];
    if ((unsigned)e < (unsigned)E) place_pair(places, p / k, p % k, e, k);
    else places.rank[p] = -1;
}

// ------------------------------------------------------------------ experts

constexpr int EX_BK = 64, EX_INFO = 4;
constexpr uint32_t EX_A_BYTES = 128 * EX_BK * 2;
constexpr int EX_DOWN_UNITS = LD / 256;

struct ExpertMaps {
    CUtensorMap gate, up, down, sh_gate, sh_up, sh_down, x, h;
};

struct Unit {
    int kind;                             // 0: gate and up, 1: down, -1: no more
    int tile, rows_at, row0, n;           // token tile, weight-row tile, first row of h and y, tokens
    int expert, t0;                       // the tile's place in the expert's list
};

template <int NT>
struct ExpertSmem {
    static constexpr uint32_t STAGE_BYTES = 2 * EX_A_BYTES + NT * EX_BK * 2;
    static constexpr int STAGES = NT <= 32 ? 5 : 4;
    // Token rows: up to eight gathers a stage by TMA, above that by four warps with
    // 16-byte asynchronous copies. (A gather of four rows holds the TMA unit as long as a
    // whole weight tile: 32 of them a stage took 4,096 tokens 504 us.)
    static constexpr bool LOADERS = NT > 32;
    // Epilogue: four warps, or eight that take every other 16 tokens (four took as long
    // for a down unit as its copies).
    static constexpr int EPI = LOADERS ? 2 : 1;
    static constexpr int THREADS = LOADERS ? 448 : 192;
    static constexpr int H_BOX = NT <= 32 ? 16 : 64;      // rows of h per copy
    alignas(1024) unsigned char stage[STAGES][STAGE_BYTES];
    alignas(8) uint64_t full[STAGES], empty[STAGES], acc_full[2], acc_empty[2], info_full[EX_INFO], info_empty[EX_INFO];
    Unit info[EX_INFO];
    int last_it[STAGES];
    int tile0[GDN_MOE_MAX_EXPERTS + 2];   // tiles before each expert (the shared one is the last), and their number
    int count[GDN_MOE_MAX_EXPERTS + 1], offset[GDN_MOE_MAX_EXPERTS + 1];
    uint32_t tmem;
    int abort;
};

__device__ __forceinline__ int load_acquire(const int *p)
{
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

// The largest exponent (biased, plus 1) of the warp's finite values: with one more in the exponent
// the others wrap round to 0.
__device__ __forceinline__ int top_exponent(float v)
{
    return (int)(__reduce_max_sync(0xffffffffu, (__float_as_uint(v) + 0x00800000u) & 0x7fffffffu) >> 23);
}

template <int NT>
__global__ void __launch_bounds__(ExpertSmem<NT>::THREADS, 1)
    moe_experts_kernel(const __grid_constant__ ExpertMaps maps, const bf16 *x, long long x_row, int M, int E, int F, int k, int shared, MoeWs ws)
{
    using Smem = ExpertSmem<NT>;
    constexpr int STAGES = Smem::STAGES;
    extern __shared__ unsigned char smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const volatile int &aborted = sm.abort;
    const int NE = E + (shared ? 1 : 0), FU = F / 128;   // experts with the shared one; gate/up units per token tile

    if (warp == 1) {
        tc::tmem_alloc(smem_u32(&sm.tmem), 4 * NT);
        tc::tmem_relinquish();
    }
    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&sm.full[s]), Smem::LOADERS ? 5 : 1);
            mbar_init(smem_u32(&sm.empty[s]), 1);
            sm.last_it[s] = -1;
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&sm.acc_full[b]), 1);
            mbar_init(smem_u32(&sm.acc_empty[b]), 4 * Smem::EPI);
        }
        for (int i = 0; i < EX_INFO; ++i) {
            mbar_init(smem_u32(&sm.info_full[i]), 1);
            mbar_init(smem_u32(&sm.info_empty[i]), Smem::LOADERS ? 13 : 5);   // warp 1, loaders, epilogue
        }
        sm.abort = 0;
        fence_mbar_init();
    }
    grid_dep_wait();
    for (int e = tid; e < NE; e += Smem::THREADS) {
        sm.count[e] = e < E ? ws.places.count[e] : M;
    }
    __syncthreads();
    if (warp == 0) {                                   // tiles and rows before each expert
        int tiles = 0, rows = 0;
        for (int e0 = 0; e0 < NE; e0 += 32) {
            const int e = e0 + lane, c = e < NE ? sm.count[e] : 0, t = (c + NT - 1) / NT;
            int ti = t, ci = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int a = __shfl_up_sync(0xffffffffu, ti, o), b = __shfl_up_sync(0xffffffffu, ci, o);
                if (lane >= o) {
                    ti += a;
                    ci += b;
                }
            }
            if (e < NE) {
                sm.tile0[e] = tiles + ti - t;
                sm.offset[e] = e < E ? rows + ci - c : M * k;
                if (blockIdx.x == 0 && e < E) ws.offset[e] = rows + ci - c;
            }
            tiles += __shfl_sync(0xffffffffu, ti, 31);
            rows += __shfl_sync(0xffffffffu, ci, 31);
        }
        if (lane == 0) sm.tile0[NE] = tiles;
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = sm.tmem;
    grid_dep_launch();

    if (warp == 0) {
        // ---- units and copies
        const int tiles = sm.tile0[NE], units1 = tiles * FU, units = units1 + tiles * EX_DOWN_UNITS;
        int it = 0, next = 0;
        // weights pass through, rows of x and h are read again (24 tokens 132 us, without this 137; 4,096 409 and 415)
        const uint64_t once = evict_first_policy();
        if (lane == 0) next = atomicAdd(ws.ticket, 1);
        for (int ui = 0;; ++ui) {
            const int u = __shfl_sync(0xffffffffu, next, 0);
            const int slot = ui % EX_INFO;
            if (ui >= EX_INFO && !mbar_wait_bounded(smem_u32(&sm.info_empty[slot]), (uint32_t)((ui / EX_INFO - 1) & 1)))
                sm.abort = 1;
            Unit un = {-1, 0, 0, 0, 0, 0, 0};
            if (!warp_gave_up(aborted) && u < units) {
                un.kind = u >= units1;
                const int per = un.kind ? EX_DOWN_UNITS : FU, v = un.kind ? u - units1 : u;
                int lo = 0, hi = NE;                   // the expert: tile0[lo] <= v / per < tile0[hi]
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (sm.tile0[mid] <= v / per) lo = mid;
                    else hi = mid;
                }
                const int e = un.expert = lo;
                const int nt = sm.tile0[e + 1] - sm.tile0[e], r = v - per * sm.tile0[e];
                un.rows_at = r / nt;
                un.t0 = (r % nt) * NT;
                un.tile = sm.tile0[e] + r % nt;
                un.row0 = sm.offset[e] + un.t0;
                un.n = min(NT, sm.count[e] - un.t0);
            }
            if (lane == 0) {
                sm.info[slot] = un;
                mbar_arrive(smem_u32(&sm.info_full[slot]));
            }
            if (un.kind < 0) break;
            if (lane == 0) next = atomicAdd(ws.ticket, 1);
            const int e = un.expert;
            const bool sh = e == E;
            const int n16 = (un.n + 15) & ~15, boxes = (un.n + Smem::H_BOX - 1) / Smem::H_BOX;
            const uint32_t bytes = 2 * EX_A_BYTES + (un.kind ? (uint32_t)(boxes * Smem::H_BOX) : Smem::LOADERS ? 0u : (uint32_t)n16) * EX_BK * 2;
            const CUtensorMap *ma, *mb;
            int ya, yb, slices;
            int4 rows = make_int4(0, 0, 0, 0);
            if (un.kind == 0) {
                ma = sh ? &maps.sh_gate : &maps.gate;
                mb = sh ? &maps.sh_up : &maps.up;
                ya = yb = (sh ? 0 : e * F) + un.rows_at * 128;
                slices = LD / EX_BK;
                if (!Smem::LOADERS && 4 * lane < n16) {   // rows past the last token repeat it
                    int r[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int t = min(4 * lane + i, un.n - 1);
                        r[i] = sh ? un.t0 + t : ws.places.token[(size_t)e * ws.places.stride + un.t0 + t];
                    }
                    rows = make_int4(r[0], r[1], r[2], r[3]);
                }
            } else {
                ma = mb = sh ? &maps.sh_down : &maps.down;
                ya = (sh ? 0 : e * LD) + un.rows_at * 256;
                yb = ya + 128;
                slices = F / EX_BK;
                if (lane == 0) {                       // the tile's h: every epilogue warp of each gate/up unit reports it
                    const uint64_t since = global_timer_ns();
                    while (load_acquire(ws.ready + un.tile) < 4 * Smem::EPI * FU) {
                        __nanosleep(100);
                        if (global_timer_ns() - since > WAIT_LIMIT_NS) {
                            sm.abort = 1;
                            break;
                        }
                    }
                }
                __syncwarp();
                fence_proxy_async_all();
            }
            for (int kb = 0; kb < slices; ++kb, ++it) {
                const int s = it % STAGES;
                if (it >= STAGES && !mbar_wait_bounded(smem_u32(&sm.empty[s]), (uint32_t)((it / STAGES - 1) & 1)))
                    sm.abort = 1;
                if (warp_gave_up(aborted)) break;
                const uint32_t dst = smem_u32(sm.stage[s]), bar = smem_u32(&sm.full[s]), b0 = dst + 2 * EX_A_BYTES;
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar, bytes);
                    tma_load_2d_hint(dst, ma, kb * EX_BK, ya, bar, once);
                    tma_load_2d_hint(dst + EX_A_BYTES, mb, kb * EX_BK, yb, bar, once);
                    sm.last_it[s] = it;
                }
                __syncwarp();
                if (un.kind == 0) {
                    if (!Smem::LOADERS && 4 * lane < n16) tma_gather4(b0 + 512u * lane, &maps.x, kb * EX_BK, rows, bar);
                } else if (lane < boxes) {
                    tma_load_2d(b0 + 128u * Smem::H_BOX * lane, &maps.h, kb * EX_BK, un.row0 + Smem::H_BOX * lane, bar);
                }
            }
        }
        if (lane == 0 && aborted)                      // copies in flight land before the CTA exits
            for (int s = 0; s < STAGES; ++s)
                if (sm.last_it[s] >= 0) mbar_wait_bounded(smem_u32(&sm.full[s]), (uint32_t)((sm.last_it[s] / STAGES) & 1));
    } else if (warp == 1) {
        // ---- products
        if (lane == 0) {
            int it = 0;
            for (int ui = 0; !aborted; ++ui) {
                const int slot = ui % EX_INFO, ab = ui & 1;
                if (!mbar_wait_bounded(smem_u32(&sm.info_full[slot]), (uint32_t)((ui / EX_INFO) & 1))) sm.abort = 1;
                if (aborted) break;
                const Unit un = sm.info[slot];
                mbar_arrive(smem_u32(&sm.info_empty[slot]));
                if (un.kind < 0) break;
                if (ui >= 2 && !mbar_wait_bounded(smem_u32(&sm.acc_empty[ab]), (uint32_t)(((ui >> 1) - 1) & 1)))
                    sm.abort = 1;
                tc::fence_after_sync();
                const uint32_t idesc = tc::instr_desc(tc::FMT_BF16, 128, (un.n + 15) & ~15);
                const uint32_t d0 = tm + (uint32_t)(2 * NT * ab), d1 = d0 + NT;
                const int slices = (un.kind ? F : LD) / EX_BK;
                for (int kb = 0; kb < slices; ++kb, ++it) {
                    const int s = it % STAGES;
                    if (!mbar_wait_bounded(smem_u32(&sm.full[s]), (uint32_t)((it / STAGES) & 1))) sm.abort = 1;
                    if (aborted) break;
                    tc::fence_after_sync();
                    const uint32_t a0 = smem_u32(sm.stage[s]);
                    const uint64_t ad = tc::sw128_desc(a0), ud = tc::sw128_desc(a0 + EX_A_BYTES);
                    const uint64_t bd = tc::sw128_desc(a0 + 2 * EX_A_BYTES);
#pragma unroll
                    for (int kk = 0; kk < EX_BK / 16; ++kk) {
                        tc::mma_f16(d0, ad + 2u * kk, bd + 2u * kk, idesc, (kb > 0 || kk > 0) ? 1u : 0u);
                        tc::mma_f16(d1, ud + 2u * kk, bd + 2u * kk, idesc, (kb > 0 || kk > 0) ? 1u : 0u);
                    }
                    tc::mma_commit(smem_u32(&sm.empty[s]));
                }
                if (aborted) break;
                tc::mma_commit(smem_u32(&sm.acc_full[ab]));
            }
        }
    } else if (warp >= 6 && warp < 10) {
        // ---- token rows (LOADERS): 8 lanes bring the 128 bytes of a row, four rows at a time. A
        //      stage is reported two slices later, when its copies have landed.
        constexpr int LAG = 2;
        const int w = warp - 6, sub = lane >> 3, chunk = lane & 7;
        int it = 0;
        auto report = [&](int i) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.full[i % STAGES]));
        };
        for (int ui = 0;; ++ui) {
            const int slot = ui % EX_INFO;
            if (!mbar_wait_sleep(smem_u32(&sm.info_full[slot]), (uint32_t)((ui / EX_INFO) & 1))) sm.abort = 1;
            if (warp_gave_up(aborted)) break;
            const Unit un = sm.info[slot];
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.info_empty[slot]));
            if (un.kind < 0) break;
            const int n16 = un.kind ? 0 : (un.n + 15) & ~15;
            const unsigned char *src[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = 32 * w + 4 * i + sub, t = min(r, un.n - 1);
                int tok = 0;
                if (r < n16) tok = un.expert == E ? un.t0 + t : ws.places.token[(size_t)un.expert * ws.places.stride + un.t0 + t];
                src[i] = reinterpret_cast<const unsigned char *>(x + (size_t)tok * x_row) + 16 * chunk;
            }
            const int slices = (un.kind ? F : LD) / EX_BK;
            for (int kb = 0; kb < slices; ++kb, ++it) {
                const int s = it % STAGES;
                if (it >= STAGES && !mbar_wait_bounded(smem_u32(&sm.empty[s]), (uint32_t)((it / STAGES - 1) & 1)))
                    sm.abort = 1;
                if (warp_gave_up(aborted)) break;
                const uint32_t b0 = smem_u32(sm.stage[s]) + 2 * EX_A_BYTES;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = 32 * w + 4 * i + sub;
                    if (r < n16) cp_async16(b0 + 128u * r + ((uint32_t)(chunk ^ (r & 7)) << 4), src[i] + 128 * kb);
                }
                cp_async_commit();
                if (it >= LAG) {
                    cp_async_wait<LAG>();
                    report(it - LAG);
                }
            }
        }
        cp_async_wait<0>();
        if (!warp_gave_up(aborted))
            for (int i = max(0, it - LAG); i < it; ++i) report(i);
    } else {
        // ---- epilogue: thread = weight row (tensor-memory lane), columns = tokens
        const int q = warp & 3, row = 32 * q + lane, c0 = warp >= 10 ? 16 : 0;
        for (int ui = 0;; ++ui) {
            const int slot = ui % EX_INFO, ab = ui & 1;
            if (!mbar_wait_sleep(smem_u32(&sm.info_full[slot]), (uint32_t)((ui / EX_INFO) & 1))) sm.abort = 1;
            if (warp_gave_up(aborted)) break;
            const Unit un = sm.info[slot];
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.info_empty[slot]));
            if (un.kind < 0) break;
            if (!mbar_wait_sleep(smem_u32(&sm.acc_full[ab]), (uint32_t)((ui >> 1) & 1))) sm.abort = 1;
            if (warp_gave_up(aborted)) break;
            tc::fence_after_sync();
            const uint32_t d0 = tc::tmem_addr(tm, 32 * q, 2 * NT * ab);
            for (int c = c0; c < un.n; c += 16 * Smem::EPI) {
                float a[16], b[16];
                tc::tmem_ld16(d0 + (uint32_t)c, a);
                tc::tmem_ld16(d0 + (uint32_t)(NT + c), b);
                tc::wait_ld();
                if (un.kind == 0) {
                    // h in bf16, as the down product takes it: 1.25e-3 of the result as a norm, where an
                    // output rounded to bf16 adds 1.65e-3
                    bf16 *p = ws.h + (size_t)(un.row0 + c) * F + un.rows_at * 128 + row;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (c + i < un.n) p[(size_t)i * F] = from_f<bf16>(silu_fast(a[i]) * b[i]);
                } else if (NT > 32) {
                    // y in 16 bits: fp16 scaled by the largest exponent among the token's 32 rows in this
                    // warp that are finite (the others stay what they are under any scale), off by at most
                    // 2^-11 of that largest value. (bf16 would add as much error as the output's own
                    // rounding; fp32 costs 2 x 150 MB at 4,096 tokens.)
                    unsigned char keep = 0;            // lane i: scale of column i, lane 16 + i: of its other block
                    __half *p = ws.y16 + (size_t)(un.row0 + c) * LD + un.rows_at * 256 + row;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int sa = max(top_exponent(a[i]), 21) - 1, sb = max(top_exponent(b[i]), 21) - 1;
                        if (lane == i) keep = (unsigned char)sa;
                        if (lane == 16 + i) keep = (unsigned char)sb;
                        if (c + i < un.n) {
                            p[(size_t)i * LD] = __float2half_rn(a[i] * __uint_as_float((uint32_t)(268 - sa) << 23));
                            p[(size_t)i * LD + 128] = __float2half_rn(b[i] * __uint_as_float((uint32_t)(268 - sb) << 23));
                        }
                    }
                    const int i = lane & 15;
                    if (c + i < un.n)
                        ws.scale[(size_t)(un.row0 + c + i) * (LD / 32) + un.rows_at * 8 + (lane >> 4) * 4 + q] = keep;
                } else {
                    float *p = ws.y + (size_t)(un.row0 + c) * LD + un.rows_at * 256 + row;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (c + i < un.n) {
                            p[(size_t)i * LD] = a[i];
                            p[(size_t)i * LD + 128] = b[i];
                        }
                }
            }
            tc::fence_before_sync();
            if (un.kind == 0) fence_proxy_async_all();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_u32(&sm.acc_empty[ab]));
                if (un.kind == 0) {
                    __threadfence();
                    asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(ws.ready + un.tile) : "memory");
                }
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) tc::tmem_dealloc(tm, 4 * NT);
    if (tid == 0 && sm.abort) atomicExch(&g_moe_error, (unsigned int)GDN_ERR_TIMEOUT);
}

// ------------------------------------------------------------------ combine

constexpr int CB_THREADS = LD / 8;

// 8 neighbouring outputs of a pair, as they are held.
template <bool Y16> struct RawY;
template <> struct RawY<false> {
    float v[8];
    __device__ __forceinline__ void load(const MoeWs &ws, size_t row, int c) { ld8(ws.y + row * LD + c, v); }
    __device__ __forceinline__ void get(float (&y)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = v[i];
    }
};
template <> struct RawY<true> {
    uint4 u;
    unsigned char scale;
    __device__ __forceinline__ void load(const MoeWs &ws, size_t row, int c)
    {
        u = *reinterpret_cast<const uint4 *>(ws.y16 + row * LD + c);
        scale = ws.scale[row * (LD / 32) + c / 32];
    }
    __device__ __forceinline__ void get(float (&y)[8]) const
    {
        const float f = __uint_as_float((uint32_t)(scale - 14) << 23);             // 2^(scale - 141)
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            y[2 * i] = v.x * f;
            y[2 * i + 1] = v.y * f;
        }
    }
};

template <typename TO, bool Y16>
__global__ void __launch_bounds__(CB_THREADS, Y16 ? 4 : 1)
    moe_combine_kernel(const bf16 *x, long long x_row, const bf16 *sh_router, const int32_t *ids, const float *weights,
                       const void *residual, void *out, int M, int k, int shared, MoeWs ws)
{
    __shared__ float part[CB_THREADS / 32], weight[GDN_MOE_MAX_TOPK];
    __shared__ int row[GDN_MOE_MAX_TOPK];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, c = tid * 8;
    const size_t m = blockIdx.x;
    grid_dep_wait();
    grid_dep_launch();
    if (tid < k) {
        const int r = ws.places.rank[m * k + tid];
        row[tid] = r < 0 ? -1 : ws.offset[ids[m * k + tid]] + r;
        weight[tid] = weights[m * k + tid];
    }
    constexpr int AHEAD = Y16 ? 8 : 4;
    float acc[8] = {};
    RawY<Y16> ys;
    if (residual) ld8(static_cast<const TO *>(residual) + m * LD + c, acc);
    if (shared) ys.load(ws, (size_t)M * k + m, c);
    float s = 0.0f;
    if (sh_router) {                                   // the shared expert's gate
        float a[8], b[8];
        ld8(x + m * x_row + c, a);
        ld8(sh_router + c, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(a[i], b[i], s);
        s = warp_sum(s);
        if (lane == 0) part[warp] = s;
    }
    __syncthreads();
    float sum[8] = {};
    for (int j = 0; j < k; j += AHEAD) {               // rows in flight, added in slot order
        RawY<Y16> y[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (j + i < k && row[j + i] >= 0) y[i].load(ws, (size_t)row[j + i], c);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (j + i < k && row[j + i] >= 0) {
                float v[8];
                y[i].get(v);
                const float w = weight[j + i];
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[e] = fmaf(w, v[e], sum[e]);
            }
    }
    if (shared) {
        float gate = 1.0f;
        if (sh_router) {
            s = 0.0f;
#pragma unroll
            for (int i = 0; i < CB_THREADS / 32; ++i) s += part[i];
            gate = 1.0f / (1.0f + expf(-s));
        }
        float y[8];
        ys.get(y);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] = fmaf(gate, y[i], sum[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] += sum[i];
    st8(static_cast<TO *>(out) + m * LD + c, acc);
}

// ------------------------------------------------------------------ launcher

static bool moe_setup()
{
    static bool ready[64] = {};
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    std::lock_guard<std::mutex> lock(mu);
    if (!ready[dev]) {
        if (cudaFuncSetAttribute(moe_experts_kernel<32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)sizeof(ExpertSmem<32>) + 1024) != cudaSuccess ||
            cudaFuncSetAttribute(moe_experts_kernel<MOE_TILE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)sizeof(ExpertSmem<MOE_TILE>) + 1024) != cudaSuccess)
            return false;
        ready[dev] = true;
    }
    return true;
}

// What a call of M tokens takes, and what every call of up to M does: rows shrink where the
// form changes, so the most is taken by M or by the last token number of a form below it.
size_t moe_call_bytes(const gdn_moe_params *p, int M) { return moe_workspace(p, M, nullptr).bytes; }
size_t moe_workspace_bytes(const gdn_moe_params *p, int M)
{
    const int last[] = {MOE_FEW_TOKENS, MOE_SMALL * p->num_experts / p->top_k};
    size_t most = moe_call_bytes(p, M);
    for (const int m : last)
        if (m < M && moe_call_bytes(p, m) > most) most = moe_call_bytes(p, m);
    return most;
}

cudaError_t launch_moe(const gdn_moe_params *p, const void *x, long long x_row, const void *residual, void *out, int M,
                       const int32_t *ids, const float *weights, void *workspace, gdn_dtype out_dt, bool lose_route, cudaStream_t s)
{
    const int n_sm = sm_count();
    if (n_sm <= 0 || !moe_setup()) return cudaErrorInvalidDevice;
    const int E = p->num_experts, F = p->ffn_dim, k = p->top_k;
    const bool shared = p->sh_gate != nullptr;
    const size_t out_row = (size_t)LD * (out_dt == GDN_F32 ? 4 : 2);
    MoeWs ws = moe_workspace(p, M, workspace);
    const bool small = moe_small(p, M);                // for the last window too: the workspace is laid out for it
    if (M <= MOE_FEW_TOKENS) return launch_moe_few(p, x, x_row, residual, out, M, ids, weights, ws, out_dt, s);
    ExpertMaps maps;
    if (!make_bf16_strided_map(&maps.gate, p->gate, (long long)E * F, LD, LD, 128) ||
        !make_bf16_strided_map(&maps.up, p->up, (long long)E * F, LD, LD, 128) ||
        !make_bf16_strided_map(&maps.down, p->down, (long long)E * LD, F, F, 128))
        return cudaErrorInvalidValue;
    if (shared && (!make_bf16_strided_map(&maps.sh_gate, p->sh_gate, F, LD, LD, 128) ||
                   !make_bf16_strided_map(&maps.sh_up, p->sh_up, F, LD, LD, 128) ||
                   !make_bf16_strided_map(&maps.sh_down, p->sh_down, LD, F, F, 128)))
        return cudaErrorInvalidValue;
    if (!shared) maps.sh_gate = maps.sh_up = maps.sh_down = maps.gate;    // not read
    for (int m0 = 0; m0 < M; m0 += MOE_WINDOW) {
        const int W = M - m0 < MOE_WINDOW ? M - m0 : MOE_WINDOW;
        const bf16 *xw = static_cast<const bf16 *>(x) + (size_t)m0 * x_row;
        const int32_t *idw = ids ? ids + (size_t)m0 * k : ws.ids;
        const float *ww = ids ? weights + (size_t)m0 * k : ws.weights;
        const size_t rows = (size_t)W * (k + (shared ? 1 : 0));
        if (!make_bf16_strided_map(&maps.x, xw, W, LD, x_row, 1) || !make_bf16_strided_map(&maps.h, ws.h, rows, F, F, small ? ExpertSmem<32>::H_BOX : ExpertSmem<MOE_TILE>::H_BOX))
            return cudaErrorInvalidValue;
        const int n_state = (int)ws.state_ints;
        cudaError_t e = cudaSuccess;
        const bool one = !ids && W <= MOE_ROUTE_TILE;  // a single cluster routes, and clears the counters itself
        if (!one) e = launch_pdl(moe_zero_kernel, dim3((n_state + 1023) / 1024), dim3(256), 0, s, ws.state, n_state);
        if (e != cudaSuccess) return e;
        e = ids ? launch_pdl(moe_place_kernel, dim3((W * k + 255) / 256), dim3(256), 0, s, idw, W * k, k, E, ws.places)
                : launch_route(p, xw, x_row, W, ws.ids, ws.weights, ws.places, one ? ws.state : nullptr, one ? n_state : 0, lose_route, s);
        if (e != cudaSuccess) return e;
        e = small ? launch_pdl(moe_experts_kernel<32>, dim3(n_sm), dim3(ExpertSmem<32>::THREADS),
                                      sizeof(ExpertSmem<32>) + 1024, s, maps, xw, x_row, W, E, F, k, (int)shared, ws)
                         : launch_pdl(moe_experts_kernel<MOE_TILE>, dim3(n_sm), dim3(ExpertSmem<MOE_TILE>::THREADS),
                                      sizeof(ExpertSmem<MOE_TILE>) + 1024, s, maps, xw, x_row, W, E, F, k, (int)shared, ws);
        if (e != cudaSuccess) return e;
        const void *rw = residual ? static_cast<const char *>(residual) + m0 * out_row : nullptr;
        void *ow = static_cast<char *>(out) + m0 * out_row;
        const bf16 *shr = static_cast<const bf16 *>(p->sh_router);
        auto combine = out_dt == GDN_F32 ? (small ? moe_combine_kernel<float, false> : moe_combine_kernel<float, true>)
                                         : (small ? moe_combine_kernel<bf16, false> : moe_combine_kernel<bf16, true>);
        e = launch_pdl(combine, dim3(W), dim3(CB_THREADS), 0, s, xw, x_row, shr, idw, ww, rw, ow, W, k, (int)shared, ws);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// Device address of this file's error word, for gdn_device_error (NULL if the lookup fails).
void *moe_error_word()
{
    void *p = nullptr;
    return cudaGetSymbolAddress(&p, g_moe_error) == cudaSuccess ? p : nullptr;
}

}  // namespace gdn
