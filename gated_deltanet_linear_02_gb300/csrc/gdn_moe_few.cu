// gdn_moe_few.cu -- the mixture-of-experts layer for at most 4 tokens, in two kernels.
// Nearly every expert that is taken has one token, so every weight is used once: a
// sweep over the weights at the rate that HBM reads, on the CUDA cores.
//  - moe_few_logits: a warp per router row (and one for the shared expert's gate),
//    all tokens.
//  - moe_few: one CTA per SM. Each chooses the experts of all tokens for itself and
//    lists the distinct ones with their tokens. Then it takes a share of the
//    (gate, up) row pairs, which its warps sweep, each with two slots of 8 KB that it keeps
//    filled by bulk copies, for h = w silu(g) * u in fp32. After that it takes a share of the
//    output dims: a producer warp brings the down rows, one expert's for all of these dims at
//    a time, while the others wait for the whole of h, whose values say themselves
//    that they are there. A CTA that has done its share of h takes another one if there is
//    any left, so that it never waits for work of a CTA that is not running.
// One token of 8 of 256 experts and a shared one: 20.9 us (8.5 at the copy's rate): 4 us logits, 4 choice
// and lists, 8 h, 1.5 until h is there, 4 outputs. Four tokens 52.8 us of 29. What it took: atomics on one address return every
// 4 ns or so, so a counter that every warp asks for each row pair cost more than the sweep;
// rows in registers instead of slots made the warps load and compute in step (3.9 TB/s);
// one producer for all row pairs fell behind (0.4 us of serial work per 8 KB).
#include <mutex>

#include "gdn_moe.cuh"
#include "gdn_route.cuh"

namespace gdn {

__device__ unsigned int g_few_error;      // GDN_ERR_TIMEOUT if a bounded wait gave up

constexpr int FW_LOGIT_WARPS = 4;
__host__ __device__ constexpr int few_logit_blocks(int experts) { return experts / FW_LOGIT_WARPS + 1; }     // of the logits and the shared expert's gate
static_assert(few_logit_blocks(GDN_MOE_MAX_EXPERTS) <= 96, "three a lane");

// What h holds until it is written: a NaN that no computation gives (a computed NaN is
// stored as another one). Reading h and waiting for it are one: no counter, no fence.
constexpr uint32_t FW_NOT_YET = 0xffffffffu;

// logits [M][E + 1], the last one the shared expert's; behind them for each token the largest sum of magnitudes of
// each CTA's experts (finite ones: the others belong to logits that are not finite either), [M][gridDim.x]
__global__ void __launch_bounds__(32 * FW_LOGIT_WARPS)
    moe_few_logits_kernel(const bf16 *x, long long x_row, const bf16 *router, const bf16 *sh_router, int M, int E,
                          int first, float *logits, int *state, uint4 *h, int h_vectors)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int e = first + blockIdx.x * FW_LOGIT_WARPS + warp;
    grid_dep_wait();
    grid_dep_launch();
    if (blockIdx.x == 0 && threadIdx.x < 2) state[threadIdx.x] = 0;
    for (int i = blockIdx.x * 32 * FW_LOGIT_WARPS + threadIdx.x; i < h_vectors; i += gridDim.x * 32 * FW_LOGIT_WARPS)
        h[i] = make_uint4(FW_NOT_YET, FW_NOT_YET, FW_NOT_YET, FW_NOT_YET);
    if (first + (int)blockIdx.x * FW_LOGIT_WARPS > E) return;
    __shared__ float mags[MOE_FEW_TOKENS][FW_LOGIT_WARPS];
    const bool there = e < E || (e == E && sh_router != nullptr);
    const bf16 *w = (e < E ? router + (size_t)e * LD : sh_router) + lane * 8;
    uint4 u[LD / 256];
#pragma unroll
    for (int c = 0; c < LD / 256; ++c) u[c] = there ? *reinterpret_cast<const uint4 *>(w + c * 256) : make_uint4(0u, 0u, 0u, 0u);
    for (int m = 0; m < M; ++m) {
        const bf16 *xm = x + (size_t)m * x_row + lane * 8;
        float s[4] = {}, t[4] = {};
#pragma unroll
        for (int c = 0; c < LD / 256; ++c) {
            float a[8], b[8];
            unpack8(u[c], a);
            ld8(xm + c * 256, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float p = __fmul_rn(a[i], b[i]);         // exact
                s[i & 3] = __fadd_rn(s[i & 3], p);
                t[i & 3] = __fadd_rn(t[i & 3], fabsf(p));
            }
        }
        const float l = warp_sum((s[0] + s[1]) + (s[2] + s[3])), mag = warp_sum((t[0] + t[1]) + (t[2] + t[3]));
        if (lane == 0) {
            if (there) logits[(size_t)m * (E + 1) + e] = l;
            mags[m][warp] = e < E && mag < INFINITY ? mag : 0.0f;
        }
    }
    __syncthreads();
    if (first == 0 && threadIdx.x < M) {               // not for a given routing
        const float *t = mags[threadIdx.x];
        logits[(size_t)M * (E + 1) + threadIdx.x * gridDim.x + blockIdx.x] = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
    }
}

// One CTA per SM, with as many warps as their slots leave room for.
constexpr int FW_MAX_WARPS = 16, FW_MIN_WARPS = 8;
constexpr uint32_t FW_SLOT = 8192;        // a row of gate and one of up; two slots a warp
constexpr int FW_ROW_SLOTS = 12;          // down rows on their way, at most, in the same memory
constexpr int FW_DIMS = 4, FW_GROUP = 4;  // output dims of a warp at a time; warps that share a group's experts
constexpr int FW_MAX_GROUPS = FW_MAX_WARPS / FW_GROUP;
constexpr int FW_POLL = 4;                // vectors of h that a thread asks for at once
constexpr int FW_MAX_PAIRS = MOE_FEW_TOKENS * (GDN_MOE_MAX_TOPK + 1);
constexpr size_t FW_SMEM_MAX = 232448 - 1024;

struct FewArgs {
    const bf16 *x, *router, *gate, *up, *down, *sh_gate, *sh_up, *sh_down;
    long long x_row;
    const int32_t *ids;                   // a given routing, or NULL
    const float *weights, *logits;
    const void *residual;
    void *out;
    float *h;                             // [M * (k + 1)][F], pair (m, j), then the shared ones
    int *state;                           // next share of h, next share of the output dims
    int M, E, F, k, renorm, sh_gated;
};

struct FewSmem {                          // behind the slots; x, then h behind it
    alignas(16) int id[FW_MAX_PAIRS];
    float weight[FW_MAX_PAIRS];
    int expert[FW_MAX_PAIRS + 1], begin[FW_MAX_PAIRS + 2];                        // distinct experts
    int pair[FW_MAX_PAIRS], token[FW_MAX_PAIRS];                                  // their pairs: h row, token
    int warp_used[RT_MAX_E / 32], warp_pairs[RT_MAX_E / 32];
    alignas(8) uint64_t full[FW_MAX_WARPS][2], row_full[FW_ROW_SLOTS], row_empty[FW_ROW_SLOTS];
    float part[FW_MAX_GROUPS][FW_DIMS * FW_GROUP][MOE_FEW_TOKENS];
    int distinct, share, dims, abort;
};

// 16 bytes of shared memory by address: shared loads whatever the compiler makes of the pointers.
__device__ __forceinline__ uint4 lds16(uint32_t addr)
{
    uint4 u;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(addr));
    return u;
}
__device__ __forceinline__ void lds8f(uint32_t addr, float (&x)[8])
{
    const uint4 a = lds16(addr), b = lds16(addr + 16);
    x[0] = __uint_as_float(a.x); x[1] = __uint_as_float(a.y); x[2] = __uint_as_float(a.z); x[3] = __uint_as_float(a.w);
    x[4] = __uint_as_float(b.x); x[5] = __uint_as_float(b.y); x[6] = __uint_as_float(b.z); x[7] = __uint_as_float(b.w);
}

// One value of h, for CTAs that poll it: a strong store, as the polls are strong loads (a weak
// one would race with them).
__device__ __forceinline__ void store_relaxed(float *p, float v)
{
    asm volatile("st.relaxed.gpu.global.f32 [%0], %1;" ::"l"(p), "f"(v) : "memory");
}

template <typename TO, bool STAGED>
__global__ void __launch_bounds__(32 * (FW_MAX_WARPS + 1), 1) moe_few_kernel(const FewArgs a)
{
    extern __shared__ unsigned char smem_raw[];
    unsigned char *ring = smem_aligned128(smem_raw);
    const int warps = (blockDim.x >> 5) - 1;              // and the producer
    FewSmem &sm = *reinterpret_cast<FewSmem *>(ring + (size_t)warps * 2 * FW_SLOT);
    unsigned char *tail = reinterpret_cast<unsigned char *>(&sm + 1);
    bf16 *xs = reinterpret_cast<bf16 *>(tail);                             // [M][2048], until h is complete
    float *hs = reinterpret_cast<float *>(tail);                           // then [M (k + 1)][F], if staged
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, threads = blockDim.x;
    const int M = a.M, F = a.F, k = a.k, P = M * k, shared = a.sh_gate != nullptr;
    const volatile int &aborted = sm.abort;
    if (tid < 2 * warps) mbar_init(smem_u32(&sm.full[0][0] + tid), 1);
    if (tid < FW_ROW_SLOTS) {
        mbar_init(smem_u32(&sm.row_full[tid]), 1);
        mbar_init(smem_u32(&sm.row_empty[tid]), FW_GROUP);
    }
    if (tid == 0) sm.abort = 0;
    fence_mbar_init();
    if (tid < 3 && shared) {                           // the shared expert's weights are needed whatever is chosen: to L2
        const size_t all = (size_t)F * LD * 2, each = (all / gridDim.x + 16) & ~(size_t)15, at = blockIdx.x * each;
        const bf16 *w = tid == 0 ? a.sh_gate : tid == 1 ? a.sh_up : a.sh_down;
        if (at < all)
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;"
                         ::"l"(reinterpret_cast<const unsigned char *>(w) + at), "r"((uint32_t)(all - at < each ? all - at : each)) : "memory");
    }
    grid_dep_wait();
    grid_dep_launch();
    if (tid == 32 * warps) {
        sm.share = atomicAdd(a.state, 1);
        sm.dims = atomicAdd(a.state + 1, 1);
    }
    for (int i = tid; i < M * (LD / 8); i += threads)
        reinterpret_cast<uint4 *>(xs)[i] = *reinterpret_cast<const uint4 *>(a.x + (size_t)(i / (LD / 8)) * a.x_row + i % (LD / 8) * 8);
    // ---- the tokens' experts
    if (a.ids) {
        if (tid < P) {
            const int e = a.ids[tid];
            sm.id[tid] = (unsigned)e < (unsigned)a.E ? e : -1;
            sm.weight[tid] = a.weights[tid];
        }
    } else if (warp < M) {
        // a logit is 23 additions deep (16 in a chain, 2, 5), each off by at most 2^-24 of its sum of
        // magnitudes: 2^-18 of the largest such sum for a difference
        float v[RT_SLOTS], mag = 0.0f, w;
        int id;
#pragma unroll
        for (int j = 0; j < RT_SLOTS; ++j) v[j] = expert_of(lane, j) < a.E ? a.logits[(size_t)warp * (a.E + 1) + expert_of(lane, j)] : 0.0f;
        const int blocks = few_logit_blocks(a.E);
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (lane + 32 * i < blocks) mag = fmaxf(mag, a.logits[(size_t)M * (a.E + 1) + warp * blocks + lane + 32 * i]);
        mag = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mag)));
        choose(v, a.E, k, a.renorm != 0, 0x1p-18f * mag, a.x + (size_t)warp * a.x_row, a.router, lane, id, w);
        if (lane < k) {
            sm.id[warp * k + lane] = id;
            sm.weight[warp * k + lane] = w;
        }
    }
    if (shared && tid >= 224 && tid < 224 + M) {       // in a warp that chooses nothing
        const int m = tid - 224;
        sm.id[P + m] = a.E;
        sm.weight[P + m] = a.sh_gated ? 1.0f / (1.0f + expf(-a.logits[(size_t)m * (a.E + 1) + a.E])) : 1.0f;
    }
    __syncthreads();
    // ---- distinct experts, the shared one first (its rows have the most tokens), and their pairs
    if (tid < RT_MAX_E) {
        int n = 0;
        for (int p = 0; p < P; ++p) n += sm.id[p] == tid;
        const uint32_t used = __ballot_sync(0xffffffffu, n > 0);
        int before = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before += t;
        }
        if (lane == 31) {
            sm.warp_used[warp] = __popc(used);
            sm.warp_pairs[warp] = before;
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
        int at = shared + __popc(used & ((1u << lane) - 1u)), first = (shared ? M : 0) + before - n, total = shared, pairs = shared ? M : 0;
        for (int w = 0; w < RT_MAX_E / 32; ++w) {
            if (w < warp) {
                at += sm.warp_used[w];
                first += sm.warp_pairs[w];
            }
            total += sm.warp_used[w];
            pairs += sm.warp_pairs[w];
        }
        if (n > 0) {
            sm.expert[at] = tid;
            sm.begin[at] = first;
            for (int p = 0; p < P; ++p)
                if (sm.id[p] == tid) {
                    sm.pair[first] = p;
                    sm.token[first++] = p / k;
                }
        }
        if (shared && tid < M) {
            sm.pair[tid] = P + tid;
            sm.token[tid] = tid;
        }
        if (tid == 0) {
            if (shared) {
                sm.expert[0] = a.E;
                sm.begin[0] = 0;
            }
            sm.begin[total] = pairs;
            sm.distinct = total;
        }
    }
    __syncthreads();
    const int distinct = sm.distinct, units = distinct * F;
    unsigned char *mine = ring + (size_t)warp * 2 * FW_SLOT;
    const uint32_t x_at = smem_u32(xs) + 16 * lane, h_at = smem_u32(hs) + 32 * lane;
    uint32_t fills = 0, reads = 0;                     // of this warp's slots, alternating: slot n & 1, phase n >> 1
    auto arrived = [&]() {
        const uint32_t n = reads++;
        if (!mbar_wait_bounded(smem_u32(&sm.full[warp][n & 1]), (n >> 1) & 1)) sm.abort = 1;
        return smem_u32(mine) + (n & 1) * FW_SLOT;
    };

    // ---- h: a row of gate and of up at a time, the experts in turn (the shared one has more
    //      tokens than the others: its rows are spread over the CTAs)
    auto fetch_pair = [&](int u) {
        if (lane == 0) {
            const int f = u / distinct, i = u - f * distinct, e = sm.expert[i];
            const bf16 *g = (e == a.E ? a.sh_gate : a.gate + (size_t)e * F * LD) + (size_t)f * LD;
            const bf16 *p = (e == a.E ? a.sh_up : a.up + (size_t)e * F * LD) + (size_t)f * LD;
            const uint32_t bar = smem_u32(&sm.full[warp][fills & 1]), dst = smem_u32(mine + (fills & 1) * FW_SLOT);
            mbar_arrive_expect_tx(bar, FW_SLOT);
            bulk_g2s(dst, g, FW_SLOT / 2, bar);
            bulk_g2s(dst + FW_SLOT / 2, p, FW_SLOT / 2, bar);
        }
        ++fills;
    };
    const int grid = gridDim.x;
    for (int share = sm.share; share < grid;) {
        const int lo = (int)((long long)units * share / grid), hi = (int)((long long)units * (share + 1) / grid);
        int more = -1;                                 // thread 0: the next share, asked for with the last row pair
        if (warp < warps) {
            if (lo + warp < hi) fetch_pair(lo + warp);
            if (lo + warp + warps < hi) fetch_pair(lo + warp + warps);
#pragma unroll 1
            for (int u = lo + warp; u < hi; u += warps) {
                if (tid == 0 && more < 0 && u + 2 * warps >= hi) more = atomicAdd(a.state, 1);
                const uint32_t slot = arrived();
                if (warp_gave_up(aborted)) break;
                const int f = u / distinct, i = u - f * distinct;
                const uint32_t gw = slot + 16 * lane;
                for (int p = sm.begin[i]; p < sm.begin[i + 1]; ++p) {
                    const int pr = sm.pair[p];
                    const uint32_t xw = x_at + sm.token[p] * (LD * 2);
                    float sg[2] = {}, su[2] = {};
#pragma unroll 4
                    for (int c = 0; c < LD / 256; ++c) {
                        float xv[8], gv[8], uv[8];
                        unpack8(lds16(xw + 512 * c), xv);
                        unpack8(lds16(gw + 512 * c), gv);
                        unpack8(lds16(gw + FW_SLOT / 2 + 512 * c), uv);
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            sg[q & 1] = fmaf(gv[q], xv[q], sg[q & 1]);
                            su[q & 1] = fmaf(uv[q], xv[q], su[q & 1]);
                        }
                    }
                    const float gs = warp_sum(sg[0] + sg[1]), us = warp_sum(su[0] + su[1]);
                    if (lane == 0) {                   // with its weight; a NaN as the common one
                        const float h = sm.weight[pr] * (silu_f(gs) * us);
                        store_relaxed(a.h + (size_t)pr * F + f, h == h ? h : __uint_as_float(0x7fffffffu));
                    }
                }
                __syncwarp();
                if (u + 2 * warps < hi) fetch_pair(u + 2 * warps);
            }
        }
        __syncthreads();
        if (tid == 0) sm.share = aborted ? grid : more < 0 ? atomicAdd(a.state, 1) : more;
        __syncthreads();
        share = sm.share;
    }
    __syncthreads();                                   // the slots and x are not needed any more

    // ---- the down rows of this CTA's output dims: at most 16 KB at a time, expert by expert. Groups
    //      of four warps take every other or every third expert, each warp four dims, and
    //      add their sums up in the end (always in the same order).
    const int d_lo = (int)((long long)LD * sm.dims / grid), d_hi = (int)((long long)LD * (sm.dims + 1) / grid);
    const int fit = (int)(2 * FW_SLOT / (2 * (uint32_t)F)), dims = min(min(fit, FW_DIMS * FW_GROUP), max(1, d_hi - d_lo));
    const int blocks = (d_hi - d_lo + dims - 1) / dims;
    const uint32_t slot_bytes = (uint32_t)dims * F * 2;
    // a multiple of the groups: a slot is always the same group's (a barrier tells a phase
    // only from the one before it)
    const int groups = warps / FW_GROUP, slots = min(FW_ROW_SLOTS, (int)((uint32_t)warps * 2 * FW_SLOT / slot_bytes)) / groups * groups;
    if (warp == warps) {
        if (lane == 0) {
            int step = 0;
            for (int b = 0; b < blocks && !aborted; ++b) {
                const int d0 = d_lo + b * dims;
                const uint32_t bytes = (uint32_t)min(dims, d_hi - d0) * F * 2;
                const size_t off = (size_t)d0 * F;
                for (int i = 0, s = step % slots; i < distinct && !aborted; ++i, ++step, s = s + 1 == slots ? 0 : s + 1) {
                    if (step >= slots && !mbar_wait_bounded(smem_u32(&sm.row_empty[s]), (uint32_t)((step / slots - 1) & 1))) {
                        sm.abort = 1;
                        break;
                    }
                    const int e = sm.expert[i];
                    const uint32_t bar = smem_u32(&sm.row_full[s]);
                    mbar_arrive_expect_tx(bar, bytes);
                    bulk_g2s(smem_u32(ring + (size_t)s * slot_bytes), (e == a.E ? a.sh_down : a.down + (size_t)e * LD * F) + off, bytes, bar);
                }
            }
            for (int n = max(0, step - slots); n < step; ++n)          // copies in flight land before the CTA exits
                mbar_wait_bounded(smem_u32(&sm.row_full[n % slots]), (uint32_t)((n / slots) & 1));
        }
    }
    // ---- all of h: into shared memory, or only waited for
    const int h_vectors = distinct == 0 ? 0 : (P + (shared ? M : 0)) * (F / 4);
    if (warp < warps)
        for (int v0 = tid; v0 < h_vectors; v0 += FW_POLL * 32 * warps) {
            uint64_t since = 0;
            uint32_t missing = 0;
#pragma unroll
            for (int j = 0; j < FW_POLL; ++j) {        // rows that nobody computes are not waited for, nor read
                const int v = v0 + j * 32 * warps;
                if (v < h_vectors && sm.id[v / (F / 4)] >= 0) missing |= 1u << j;
            }
            while (missing && !aborted) {
                uint4 r[FW_POLL];
#pragma unroll
                for (int j = 0; j < FW_POLL; ++j)
                    if (missing >> j & 1u)
                        asm volatile("ld.relaxed.gpu.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(r[j].x), "=r"(r[j].y), "=r"(r[j].z), "=r"(r[j].w)
                                     : "l"(reinterpret_cast<const uint4 *>(a.h) + v0 + j * 32 * warps) : "memory");
#pragma unroll
                for (int j = 0; j < FW_POLL; ++j)
                    if ((missing >> j & 1u) && r[j].x != FW_NOT_YET && r[j].y != FW_NOT_YET && r[j].z != FW_NOT_YET &&
                        r[j].w != FW_NOT_YET) {
                        if (STAGED) reinterpret_cast<uint4 *>(hs)[v0 + j * 32 * warps] = r[j];
                        missing &= ~(1u << j);
                    }
                if (since == 0) since = global_timer_ns();
                else if (missing && global_timer_ns() - since > WAIT_LIMIT_NS) sm.abort = 1;
            }
        }
    if (warp < warps) {
        if (!STAGED) __threadfence();
        __syncwarp();
        asm volatile("bar.sync 2, %0;" ::"r"(32 * warps) : "memory");
        // ---- output dims; a lane keeps its share of every token's sums
        const int group = warp / FW_GROUP, row0 = (warp % FW_GROUP) * FW_DIMS;
        int step = 0;
        for (int b = 0; b < blocks; ++b) {
            const int d0 = d_lo + b * dims, n = min(dims, d_hi - d0);
            float acc[FW_DIMS][MOE_FEW_TOKENS] = {};
            if (group < groups)
                for (int i = (group + groups - step % groups) % groups; i < distinct; i += groups) {
                    const int q = step + i, s = q % slots;
                    if (!mbar_wait_bounded(smem_u32(&sm.row_full[s]), (uint32_t)((q / slots) & 1))) sm.abort = 1;
                    if (warp_gave_up(aborted)) break;
                    const uint32_t rows = smem_u32(ring) + s * slot_bytes + (uint32_t)(row0 * F + lane * 8) * 2;
                    for (int p = sm.begin[i]; p < sm.begin[i + 1]; ++p) {
                        const int at = sm.pair[p] * F, m = sm.token[p];
                        float sum[FW_DIMS][2] = {};
#pragma unroll 1
                        for (int c = 0; c < F; c += 256) {
                            if (c + lane * 8 >= F) break;
                            float hv[8];
                            if (STAGED) lds8f(h_at + (at + c) * 4, hv);
                            else ld8(a.h + (size_t)at + c + lane * 8, hv);
#pragma unroll
                            for (int r = 0; r < FW_DIMS; ++r) {        // rows past n: in the slots, and not used
                                float wv[8];
                                unpack8(lds16(rows + (uint32_t)(min(r, n - 1 - row0) * F + c) * 2), wv);
#pragma unroll
                                for (int t = 0; t < 8; ++t) sum[r][t & 1] = fmaf(wv[t], hv[t], sum[r][t & 1]);
                            }
                        }
#pragma unroll
                        for (int r = 0; r < FW_DIMS; ++r)
#pragma unroll
                            for (int t = 0; t < MOE_FEW_TOKENS; ++t) acc[r][t] += t == m ? sum[r][0] + sum[r][1] : 0.0f;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sm.row_empty[s]));
                }
            if (group < groups) {
#pragma unroll
                for (int r = 0; r < FW_DIMS; ++r)
#pragma unroll
                    for (int m = 0; m < MOE_FEW_TOKENS; ++m) {
                        const float sum = warp_sum(acc[r][m]);
                        if (lane == 0) sm.part[group][row0 + r][m] = sum;
                    }
            }
            asm volatile("bar.sync 2, %0;" ::"r"(32 * warps) : "memory");
            if (tid < n * M) {
                const int j = tid % n, m = tid / n;
                const size_t at = (size_t)m * LD + d0 + j;
                float sum = 0.0f;
                for (int g = 0; g < groups; ++g) sum += sm.part[g][j][m];
                if (a.residual) sum += to_f(static_cast<const TO *>(a.residual)[at]);
                if (!aborted) static_cast<TO *>(a.out)[at] = from_f<TO>(sum);
            }
            asm volatile("bar.sync 2, %0;" ::"r"(32 * warps) : "memory");
            step += distinct;
        }
        if (aborted) {                                 // copies in flight land before the CTA exits
            while (reads < fills) {
                const uint32_t n = reads++;
                mbar_wait_bounded(smem_u32(&sm.full[warp][n & 1]), (n >> 1) & 1);
            }
            if (lane == 0) atomicExch(&g_few_error, (unsigned int)GDN_ERR_TIMEOUT);
        }
    }
}

static bool few_setup()
{
    static bool ready[64] = {};
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    std::lock_guard<std::mutex> lock(mu);
    if (!ready[dev]) {
        const int n = (int)FW_SMEM_MAX;
        const cudaFuncAttribute at = cudaFuncAttributeMaxDynamicSharedMemorySize;
        if (cudaFuncSetAttribute(moe_few_kernel<float, true>, at, n) != cudaSuccess ||
            cudaFuncSetAttribute(moe_few_kernel<float, false>, at, n) != cudaSuccess ||
            cudaFuncSetAttribute(moe_few_kernel<bf16, true>, at, n) != cudaSuccess ||
            cudaFuncSetAttribute(moe_few_kernel<bf16, false>, at, n) != cudaSuccess)
            return false;
        ready[dev] = true;
    }
    return true;
}

cudaError_t launch_moe_few(const gdn_moe_params *p, const void *x, long long x_row, const void *residual, void *out, int M,
                           const int32_t *ids, const float *weights, const MoeWs &ws, gdn_dtype out_dt, cudaStream_t s)
{
    const int n_sm = sm_count();
    if (n_sm <= 0 || !few_setup()) return cudaErrorInvalidDevice;
    const int E = p->num_experts, first = ids ? E : 0;          // with a given routing only the shared expert's gate
    cudaError_t e = launch_pdl(moe_few_logits_kernel, dim3(ids ? 32 : few_logit_blocks(E)),
                               dim3(32 * FW_LOGIT_WARPS), 0, s, (const bf16 *)x, x_row, (const bf16 *)p->router,
                               (const bf16 *)p->sh_router, M, E, first, ws.logits, ws.state, (uint4 *)ws.y,
                               M * (p->top_k + (p->sh_gate ? 1 : 0)) * (p->ffn_dim / 4));
    if (e != cudaSuccess) return e;
    FewArgs a = {};
    a.x = (const bf16 *)x; a.router = (const bf16 *)p->router;
    a.gate = (const bf16 *)p->gate; a.up = (const bf16 *)p->up; a.down = (const bf16 *)p->down;
    a.sh_gate = (const bf16 *)p->sh_gate; a.sh_up = (const bf16 *)p->sh_up; a.sh_down = (const bf16 *)p->sh_down;
    a.x_row = x_row; a.ids = ids; a.weights = weights; a.logits = ws.logits; a.residual = residual; a.out = out;
    a.h = ws.y; a.state = ws.state; a.M = M; a.E = E; a.F = p->ffn_dim; a.k = p->top_k; a.renorm = p->norm_topk;
    a.sh_gated = p->sh_router != nullptr;
    // Shared memory: two slots a warp, then x and, in its place later, h where it leaves room
    // for 8 warps (else h is read from global memory).
    const size_t xb = (size_t)M * LD * 2, hb = (size_t)M * (a.k + (a.sh_gate ? 1 : 0)) * a.F * 4, base = sizeof(FewSmem) + 128;
    const bool staged = base + (hb > xb ? hb : xb) + FW_MIN_WARPS * 2 * FW_SLOT <= FW_SMEM_MAX;
    const size_t fixed = base + (staged && hb > xb ? hb : xb);
    int warps = (int)((FW_SMEM_MAX - fixed) / (2 * FW_SLOT));
    if (warps > FW_MAX_WARPS) warps = FW_MAX_WARPS;
    const size_t smem = fixed + (size_t)warps * 2 * FW_SLOT;
    const dim3 g(n_sm), b(32 * (warps + 1));
    if (out_dt == GDN_F32)
        return staged ? launch_pdl(moe_few_kernel<float, true>, g, b, smem, s, a) : launch_pdl(moe_few_kernel<float, false>, g, b, smem, s, a);
    return staged ? launch_pdl(moe_few_kernel<bf16, true>, g, b, smem, s, a) : launch_pdl(moe_few_kernel<bf16, false>, g, b, smem, s, a);
}

// Device address of this file's error word, for gdn_device_error (NULL if the lookup fails).
void *few_error_word()
{
    void *p = nullptr;
    return cudaGetSymbolAddress(&p, g_few_error) == cudaSuccess ? p : nullptr;
}

}  // namespace gdn
