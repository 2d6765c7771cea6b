// gdn_linear.cu -- y = residual + act(x w^T + bias) on 5th-generation tensor cores:
// bf16 operands, fp32 accumulation, everything behind the product in the
// epilogue, on the fp32 accumulators, with one rounding at the end. The dense
// products of "qwen35moe -- Forward-Pass Design (Pantheon port)" that have no
// entry point of their own: steps 1 and 7 of section "Full-attention block"
// (joint query and gate, key and value projection; attn_output with the residual).
//
// Two forms:
//  - pair_kernel, for many rows: pairs of CTAs (cta_group::2) take 256 x BN tiles (BN = 256,
//    or 128 where those are too few), each CTA 128 rows of x and half of the
//    columns' weights, so that an operand byte in shared memory serves twice the products of
//    a lone CTA (whose 128 x 256 tiles run into the shared-memory port at 1.45
//    PFLOP/s). A TMA warp in each CTA, one issuing thread in the leader, eight epilogue
//    warps in each, two accumulators in tensor memory.
//  - linear_kernel, for few rows: tiles of 128 rows x 128 columns, each tile's K range
//    split over the CTAs of a cluster, whose partial tiles meet in distributed
//    shared memory (always in the same order).
// 4,001 x 9,216 x 2,048 with bias and SiLU: 104 us, 1.45 PFLOP/s; 93 to 96 us in short runs, before
// power caps the clock, where it is bound by what L2 brings to the SMs (12.7 TB/s). 8,192^3, short
// runs: 1.73 PFLOP/s. One row, 2,048 -> 9,216: 9.8 us (3.8 TB/s), 4,096 -> 2,048: 6.3 us; there the start,
// the issue of the products and the cluster's exchange bind. Between 129 and some 3,000 rows tiles are few
// and whole waves of them are half empty: 768 x 2,048 x 4,096 19.8 us.
#include <mutex>

#include "gdn_layer.cuh"
#include "gdn_tc.cuh"
#include "gdn_tma.cuh"

namespace gdn {

__device__ unsigned int g_linear_error;   // GDN_ERR_TIMEOUT if a bounded wait gave up

constexpr int LN_BM = 128, LN_BK = 64, LN_THREADS = 192;
constexpr uint32_t LN_A_BYTES = LN_BM * LN_BK * 2;

struct LinearOut {
    const float *bias;
    const void *residual;
    void *y;
    long long r_row, y_row;
};

// v / 2 * erfc(-v / sqrt 2) for any v, relative to its value (1 + erf cancels for negative v, and is 0
// from -5.5 on). With t = |v| / sqrt 2, in the form of Hastings' approximations (Abramowitz and
// Stegun 7.1.26): erfc(t) = exp(-t^2) u q(u), u = 1 / (1 + 0.55 t), which brings t in [0, inf) to (0, 1].
// q is a polynomial of degree 9 fitted here, least squares on exp(t^2) erfc(t) / u over |v| <= 14 with
// weights that even the relative error out (below 2^-27). exp(-v^2 / 2) by the special function (its
// argument is off by v^2 2^-24), u with a Newton step behind it. 4,001 x 9,216 x 2,048: 99 us;
// with erfcf 133, with 1 + erff 102.
__device__ __forceinline__ float gelu(float v)
{
    const float a = fminf(fabsf(v), 14.0f);            // NaN comes back with the product below
    const float d = fmaf(a, 0.38890874f, 1.0f);
    float u, e;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(u) : "f"(d));
    u = fmaf(u, fmaf(-d, u, 1.0f), u);
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(a * a * -0.72134752044448170f));
    float q = 0.029023804f;                            // half of q's coefficients
    q = fmaf(q, u, -0.16832937f);
    q = fmaf(q, u, 0.39062503f);
    q = fmaf(q, u, -0.42671686f);
    q = fmaf(q, u, 0.18198204f);
    q = fmaf(q, u, -0.047497895f);
    q = fmaf(q, u, 0.10102546f);
    q = fmaf(q, u, 0.12940997f);
    q = fmaf(q, u, 0.15533178f);
    q = fmaf(q, u, 0.15514605f);
    const float h = q * u * e;                         // erfc(t) / 2
    return v * (v < 0.0f ? h : 1.0f - h);
}

// For bf16 outputs exp and the division by special functions, whose error grows with |v|, by
// 2^-23 (4 + 2 |v|) of the value at most, far below the output's rounding; 0 where the denominator
// passes 2^126 (silu and sigmoid below -87.3). For fp32 outputs within 2^-21 down to fp32's last
// numbers, by exp(-|v|), which does not overflow. 4,001 x 9,216 x 2,048 with SiLU to
// fp32: 128 us (with the functions of bf16 127), 96 rows 13.1 (13.0).
template <typename TO, int ACT>
__device__ __forceinline__ float apply_act(float v)
{
    if (ACT == GDN_ACT_GELU) return gelu(v);
    if (ACT == GDN_ACT_NONE) return v;
    const float top = ACT == GDN_ACT_SILU ? v : 1.0f;
    if (sizeof(TO) == 2) return __fdividef(top, 1.0f + __expf(-v));
    const float e = expf(-fabsf(v));
    return top * __fdividef(v < 0.0f ? e : 1.0f, 1.0f + e);         // the denominator is at most 2
}

// Brings the tensor maps near before the first copies need them.
__device__ __forceinline__ void prefetch_maps(const CUtensorMap *a, const CUtensorMap *b)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(a)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(b)) : "memory");
}

// Epilogue of NC (8 or 32) neighbouring columns of row m, those below N; loads first.
template <typename TO, int ACT, int NC>
__device__ __forceinline__ void finish(const LinearOut &o, int m, int n, int N, float (&v)[NC])
{
    float r[NC], b[NC];
    if (o.residual)
#pragma unroll
        for (int e = 0; e < NC; e += 8)
            if (n + e < N) ld8(static_cast<const TO *>(o.residual) + (size_t)m * o.r_row + n + e, reinterpret_cast<float(&)[8]>(r[e]));
    if (o.bias)
#pragma unroll
        for (int e = 0; e < NC; e += 8)
            if (n + e < N) ld8(o.bias + n + e, reinterpret_cast<float(&)[8]>(b[e]));
    if (o.bias)
#pragma unroll
        for (int i = 0; i < NC; ++i) v[i] += b[i];
    if (ACT != GDN_ACT_NONE)
#pragma unroll
        for (int i = 0; i < NC; ++i) v[i] = apply_act<TO, ACT>(v[i]);
    if (o.residual)
#pragma unroll
        for (int i = 0; i < NC; ++i) v[i] += r[i];
#pragma unroll
    for (int e = 0; e < NC; e += 8)
        if (n + e < N) st8(static_cast<TO *>(o.y) + (size_t)m * o.y_row + n + e, reinterpret_cast<float(&)[8]>(v[e]));
}

// ------------------------------------------------------------------ many rows: pairs of CTAs

// Forms of the tensor-core and copy instructions for a pair of CTAs.
__device__ __forceinline__ void pair_tmem_alloc(uint32_t smem_dst, uint32_t ncols)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_dst), "r"(ncols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_tmem_dealloc(uint32_t taddr, uint32_t ncols)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}
// Arrives once on the barrier at this offset in both CTAs when the products so far are done.
__device__ __forceinline__ void pair_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 ::"r"(bar), "h"((uint16_t)3) : "memory");
}
// A box into this CTA's shared memory, counted on a barrier of the leader.
__device__ __forceinline__ void pair_load_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t leader_bar)
{
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3}], [%4];"
                 ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(leader_bar) : "memory");
}
// Only reads of tensor memory come before it, which tcgen05's own fences order: at
// cluster scope it would wait for the epilogue's stores.
__device__ __forceinline__ void arrive_cluster(uint32_t cluster_bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
constexpr int PR_THREADS = 320;           // TMA warp, MMA warp, eight epilogue warps

// A stage holds two slices of 64 along K: eight products for one wait and one commit. (With one
// slice a stage the issuing thread took 720 cycles for 512 of arithmetic.)
template <int BN>
struct PairSmem {
    static constexpr int STAGES = BN == 256 ? 3 : 4;
    static constexpr uint32_t SLICE_BYTES = LN_A_BYTES + BN / 2 * LN_BK * 2, STAGE_BYTES = 2 * SLICE_BYTES;
    alignas(1024) unsigned char stage[STAGES][STAGE_BYTES];
    alignas(8) uint64_t full[STAGES], empty[STAGES], acc_full[2], acc_empty[2];
    int last_it[STAGES];
    uint32_t tmem;
    int abort;
};

template <typename TO, int BN, int ACT>
__global__ void __launch_bounds__(PR_THREADS, 1)
    pair_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw, const LinearOut out, int M,
                int N, int K)
{
    using Smem = PairSmem<BN>;
    constexpr int STAGES = Smem::STAGES;
    extern __shared__ unsigned char smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)blockIdx.x & 1, pair = (int)blockIdx.x >> 1, pairs = (int)gridDim.x >> 1;
    const int m_tiles = (M + 255) / 256, tiles = m_tiles * ((N + BN - 1) / BN), slices = (K + LN_BK - 1) / LN_BK;
    const volatile int &aborted = sm.abort;

    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&sm.full[s]), 1);
            mbar_init(smem_u32(&sm.empty[s]), 1);
            sm.last_it[s] = -1;
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&sm.acc_full[b]), 1);
            mbar_init(smem_u32(&sm.acc_empty[b]), 16);             // the epilogue warps of both CTAs
        }
        sm.abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) pair_tmem_alloc(smem_u32(&sm.tmem), 2 * BN);
    if (tid == 64) prefetch_maps(&mx, &mw);
    tc::fence_before_sync();
    __syncthreads();
    cluster_sync_all();                                // both CTAs' barriers exist
    tc::fence_after_sync();
    const uint32_t tm = sm.tmem;
    grid_dep_wait();
    grid_dep_launch();

    if (warp == 0) {
        if (lane == 0) {
            int it = 0;
            for (int t = pair; t < tiles && !aborted; t += pairs) {
                const int mt = t % m_tiles, nt = t / m_tiles;
                for (int kb = 0; kb < slices; kb += 2, ++it) {
                    const int s = it % STAGES, two = kb + 1 < slices;
                    if (it >= STAGES && !mbar_wait_bounded(smem_u32(&sm.empty[s]), (uint32_t)((it / STAGES - 1) & 1))) sm.abort = 1;
                    if (aborted) break;
                    const uint32_t dst = smem_u32(sm.stage[s]), bar = mapa_shared(smem_u32(&sm.full[s]), 0);
                    if (rank == 0) mbar_arrive_expect_tx(smem_u32(&sm.full[s]), 2 * Smem::SLICE_BYTES * (1 + two));
                    for (int h = 0; h <= two; ++h) {
                        const uint32_t at = dst + h * Smem::SLICE_BYTES;
                        pair_load_2d(at, &mx, (kb + h) * LN_BK, mt * 256 + rank * 128, bar);
                        pair_load_2d(at + LN_A_BYTES, &mw, (kb + h) * LN_BK, nt * BN + rank * (BN / 2), bar);
                    }
                    sm.last_it[s] = it;
                }
            }
            // every copy of the pair has landed before its CTAs leave: the leader waits, its partner meets it below
            if (rank == 0)
                for (int s = 0; s < STAGES; ++s)
                    if (sm.last_it[s] >= 0 && !mbar_wait_bounded(smem_u32(&sm.full[s]), (uint32_t)((sm.last_it[s] / STAGES) & 1)))
                        sm.abort = 1;
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            const uint32_t idesc = tc::instr_desc(tc::FMT_BF16, 256, BN);
            int it = 0, ti = 0;
            for (int t = pair; t < tiles && !aborted; t += pairs, ++ti) {
                const int ab = ti & 1;
                if (ti >= 2 && !mbar_wait_bounded(smem_u32(&sm.acc_empty[ab]), (uint32_t)(((ti >> 1) - 1) & 1))) sm.abort = 1;
                tc::fence_after_sync();
                const uint32_t d = tm + (uint32_t)(BN * ab);
                for (int kb = 0; kb < slices; kb += 2, ++it) {
                    const int s = it % STAGES, two = kb + 1 < slices;
                    if (!mbar_wait_bounded(smem_u32(&sm.full[s]), (uint32_t)((it / STAGES) & 1))) sm.abort = 1;
                    if (aborted) break;
                    tc::fence_after_sync();
                    const uint64_t ad = tc::sw128_desc(smem_u32(sm.stage[s]));
                    const uint64_t bd = tc::sw128_desc(smem_u32(sm.stage[s]) + LN_A_BYTES);
#pragma unroll
                    for (int k = 0; k < LN_BK / 16; ++k)
                        pair_mma(d, ad + 2u * k, bd + 2u * k, idesc, (kb > 0 || k > 0) ? 1u : 0u);
                    if (two) {
#pragma unroll
                        for (int k = 0; k < LN_BK / 16; ++k)
                            pair_mma(d, ad + (Smem::SLICE_BYTES >> 4) + 2u * k, bd + (Smem::SLICE_BYTES >> 4) + 2u * k, idesc, 1u);
                    }
                    pair_commit(smem_u32(&sm.empty[s]));
                }
                if (aborted) break;
                pair_commit(smem_u32(&sm.acc_full[ab]));
            }
        }
    } else {
        const int q = warp & 3, half = (warp - 2) >> 2;                // lanes 32 q.., half of the columns
        int ti = 0;
        for (int t = pair; t < tiles; t += pairs, ++ti) {
            const int ab = ti & 1, mt = t % m_tiles, nt = t / m_tiles;
            if (!mbar_wait_bounded(smem_u32(&sm.acc_full[ab]), (uint32_t)((ti >> 1) & 1))) sm.abort = 1;
            if (warp_gave_up(aborted)) break;
            tc::fence_after_sync();
            const int m = mt * 256 + rank * 128 + 32 * q + lane;
#pragma unroll 1
            for (int c = half * (BN / 2); c < (half + 1) * (BN / 2); c += 32) {
                float v[32];
                tc::tmem_ld32(tc::tmem_addr(tm + (uint32_t)(BN * ab), 32 * q, c), v);
                tc::wait_ld();
                if (m < M) finish<TO, ACT, 32>(out, m, nt * BN + c, N, v);
                __syncwarp();
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) arrive_cluster(mapa_shared(smem_u32(&sm.acc_empty[ab]), 0));
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    cluster_sync_all();                                // nobody's barriers or tensor memory are used any more
    tc::fence_after_sync();
    if (warp == 1) pair_tmem_dealloc(tm, 2 * BN);
    if (tid == 0 && sm.abort) atomicExch(&g_linear_error, (unsigned int)GDN_ERR_TIMEOUT);
}

// ------------------------------------------------------------------ few rows: split K

constexpr int LN_BN = 128, LN_MAX_STAGES = 6, LN_PART_LD = LN_BN + 4;
constexpr uint32_t LN_B_BYTES = LN_BN * LN_BK * 2;
constexpr uint32_t LN_RING = 212 * 1024;  // stages, with 16 KB behind the last one that a short A tile's products may read
static_assert(LN_BM * LN_PART_LD * 4 <= LN_RING, "a partial tile fits the stages");

struct LinearSmem {
    alignas(1024) unsigned char ring[LN_RING];
    alignas(8) uint64_t full[LN_MAX_STAGES], empty[LN_MAX_STAGES], acc_full[2], acc_empty[2];
    int last_round[LN_MAX_STAGES];
    uint32_t tmem;
    int abort;
};

// The sums of a cluster's partial tiles for rows [r0, r0 + rows) of this CTA's tile: each
// of 128 threads takes every 128th group of 8 columns, U groups at a time with all their
// remote loads in flight, S >= splits.
template <typename TO, int ACT, int S, int U>
__device__ __forceinline__ void add_partials(const LinearOut &out, uint32_t part0, int splits, int r0, int rows, int m0,
                                             int n0, int N, int t)
{
    constexpr int GROUPS = LN_BN / 8;
    for (int f0 = t; f0 < rows * GROUPS; f0 += 128 * U) {
        float4 a[U][S], b[U][S];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int f = f0 + 128 * u, rr = r0 + f / GROUPS, col = 8 * (f % GROUPS);
            if (f < rows * GROUPS && n0 + col < N) {
#pragma unroll
                for (int r = 0; r < S; ++r)
                    if (r < splits) {
                        const uint32_t at = mapa_shared(part0 + (uint32_t)((rr * LN_PART_LD + col) * 4), (uint32_t)r);
                        a[u][r] = ld_cluster_f32x4(at);
                        b[u][r] = ld_cluster_f32x4(at + 16);
                    }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int f = f0 + 128 * u, rr = r0 + f / GROUPS, col = 8 * (f % GROUPS);
            if (f < rows * GROUPS && n0 + col < N) {
                float v[8] = {a[u][0].x, a[u][0].y, a[u][0].z, a[u][0].w, b[u][0].x, b[u][0].y, b[u][0].z, b[u][0].w};
#pragma unroll
                for (int r = 1; r < S; ++r)
                    if (r < splits) {
                        v[0] += a[u][r].x; v[1] += a[u][r].y; v[2] += a[u][r].z; v[3] += a[u][r].w;
                        v[4] += b[u][r].x; v[5] += b[u][r].y; v[6] += b[u][r].z; v[7] += b[u][r].w;
                    }
                finish<TO, ACT, 8>(out, m0 + rr, n0 + col, N, v);
            }
        }
    }
}

// a_rows: rows of x that a stage holds, 128, or with fewer rows in all those, rounded up
// to 8; two slices of 64 along K a stage, as above. The products read 128 rows all the same; what the others hold does not
// matter, as each row of the tile has its own sums. Shorter stages, more of them:
// more weights in flight.
template <typename TO, int ACT>
__global__ void __launch_bounds__(LN_THREADS, 1)
    linear_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw, const LinearOut out,
                  int M, int N, int K, int splits, int a_rows, int STAGES)
{
    constexpr int BN = LN_BN, PLD = LN_PART_LD;
    extern __shared__ unsigned char smem_raw[];
    LinearSmem &sm = *reinterpret_cast<LinearSmem *>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
    const uint32_t a_bytes = (uint32_t)a_rows * LN_BK * 2, slice_bytes = a_bytes + LN_B_BYTES, stage_bytes = 2 * slice_bytes, ring = smem_u32(sm.ring);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n_tiles = (N + BN - 1) / BN;
    const bool split = splits > 1;
    const int w0 = split ? (int)blockIdx.x / splits : (int)blockIdx.x;
    const int wstep = split ? 1 : (int)gridDim.x;
    const int wend = split ? w0 + 1 : ((M + LN_BM - 1) / LN_BM) * n_tiles;
    const int kb_all = (K + LN_BK - 1) / LN_BK, part = split ? (int)blockIdx.x % splits : 0;
    const int kb0 = kb_all * part / splits, kb1 = kb_all * (part + 1) / splits;   // never empty: splits <= kb_all
    const volatile int &aborted = sm.abort;

    if (warp == 1) {
        tc::tmem_alloc(smem_u32(&sm.tmem), 2 * BN);
        tc::tmem_relinquish();
    }
    if (tid == 64) prefetch_maps(&mx, &mw);
    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&sm.full[s]), 1);
            mbar_init(smem_u32(&sm.empty[s]), 1);
            sm.last_round[s] = -1;
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&sm.acc_full[b]), 1);
            mbar_init(smem_u32(&sm.acc_empty[b]), 128);
        }
        sm.abort = 0;
        fence_mbar_init();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = sm.tmem;
    grid_dep_wait();
    grid_dep_launch();

    if (warp == 0) {
        if (lane == 0) {
            int s = 0, round = 0;                      // stage, and how often the ring has gone round
            for (int w = w0; w < wend && !aborted; w += wstep) {
                const int mt = w / n_tiles, nt = w % n_tiles;
                for (int kb = kb0; kb < kb1; kb += 2) {
                    if (round > 0 && !mbar_wait_bounded(smem_u32(&sm.empty[s]), (uint32_t)((round - 1) & 1))) sm.abort = 1;
                    if (aborted) break;
                    const int two = kb + 1 < kb1;
                    const uint32_t dst = ring + s * stage_bytes, bar = smem_u32(&sm.full[s]);
                    mbar_arrive_expect_tx(bar, slice_bytes * (1 + two));
                    for (int h = 0; h <= two; ++h) {
                        tma_load_2d(dst + h * slice_bytes + a_bytes, &mw, (kb + h) * LN_BK, nt * BN, bar);
                        tma_load_2d(dst + h * slice_bytes, &mx, (kb + h) * LN_BK, mt * LN_BM, bar);
                    }
                    sm.last_round[s] = round;
                    if (++s == STAGES) {
                        s = 0;
                        ++round;
                    }
                }
            }
            if (aborted)                               // copies in flight land before the CTA exits
                for (s = 0; s < STAGES; ++s)
                    if (sm.last_round[s] >= 0) mbar_wait_bounded(smem_u32(&sm.full[s]), (uint32_t)(sm.last_round[s] & 1));
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = tc::instr_desc(tc::FMT_BF16, LN_BM, BN);
            int s = 0, round = 0, ti = 0;
            for (int w = w0; w < wend && !aborted; w += wstep, ++ti) {
                const int ab = ti & 1;
                if (ti >= 2 && !mbar_wait_bounded(smem_u32(&sm.acc_empty[ab]), (uint32_t)(((ti >> 1) - 1) & 1)))
                    sm.abort = 1;
                tc::fence_after_sync();
                const uint32_t d = tm + (uint32_t)(BN * ab);
                for (int kb = kb0; kb < kb1; kb += 2) {
                    if (!mbar_wait_bounded(smem_u32(&sm.full[s]), (uint32_t)(round & 1))) sm.abort = 1;
                    if (aborted) break;
                    tc::fence_after_sync();
                    const uint64_t ad = tc::sw128_desc(ring + s * stage_bytes), bd = tc::sw128_desc(ring + s * stage_bytes + a_bytes);
#pragma unroll
                    for (int k = 0; k < LN_BK / 16; ++k)
                        tc::mma_f16(d, ad + 2u * k, bd + 2u * k, idesc, (kb > kb0 || k > 0) ? 1u : 0u);
                    if (kb + 1 < kb1) {
#pragma unroll
                        for (int k = 0; k < LN_BK / 16; ++k)
                            tc::mma_f16(d, ad + (slice_bytes >> 4) + 2u * k, bd + (slice_bytes >> 4) + 2u * k, idesc, 1u);
                    }
                    tc::mma_commit(smem_u32(&sm.empty[s]));
                    if (++s == STAGES) {
                        s = 0;
                        ++round;
                    }
                }
                if (aborted) break;
                tc::mma_commit(smem_u32(&sm.acc_full[ab]));
            }
        }
    } else {
        const int q = warp & 3, row = 32 * q + lane;
        if (split) {                                   // this CTA's fp32 partial tile into shared memory
            if (!mbar_wait_bounded(smem_u32(&sm.acc_full[0]), 0)) sm.abort = 1;
            __syncwarp();
            tc::fence_after_sync();
            float *p = reinterpret_cast<float *>(sm.ring) + row * PLD;
            const bool some = (w0 / n_tiles) * LN_BM + 32 * q < M;     // of this warp's rows
            for (int c = 0; c < BN && some; c += 32) {
                float v[32];
                tc::tmem_ld32(tc::tmem_addr(tm, 32 * q, c), v);
                tc::wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    reinterpret_cast<float4 *>(p + c)[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
            }
        }
        int ti = 0;
        for (int w = w0; w < wend && !split; w += wstep, ++ti) {
            const int ab = ti & 1, mt = w / n_tiles, nt = w % n_tiles;
            if (!mbar_wait_bounded(smem_u32(&sm.acc_full[ab]), (uint32_t)((ti >> 1) & 1))) sm.abort = 1;
            if (warp_gave_up(aborted)) break;          // tensor memory is read by whole warps
            tc::fence_after_sync();
            const int m = mt * LN_BM + row;
            for (int c = 0; c < BN; c += 32) {
                float v[32];
                tc::tmem_ld32(tc::tmem_addr(tm + (uint32_t)(BN * ab), 32 * q, c), v);
                tc::wait_ld();
                const int n = nt * BN + c;
                if (m < M) finish<TO, ACT, 32>(out, m, n, N, v);
                __syncwarp();
            }
            tc::fence_before_sync();
            mbar_arrive(smem_u32(&sm.acc_empty[ab]));
        }
    }
    if (split) {
        // each CTA of the cluster writes an even share of the tile's rows, each the sum of the S partials
        cluster_sync_all();
        if (warp >= 2 && !aborted) {
            const int mt = w0 / n_tiles, nt = w0 % n_tiles, there = min(LN_BM, M - mt * LN_BM);
            const int r0 = there * part / splits, rows = there * (part + 1) / splits - r0;
            if (splits <= 2) add_partials<TO, ACT, 2, 4>(out, ring, splits, r0, rows, mt * LN_BM, nt * BN, N, tid - 64);
            else if (splits <= 4) add_partials<TO, ACT, 4, 2>(out, ring, splits, r0, rows, mt * LN_BM, nt * BN, N, tid - 64);
            else add_partials<TO, ACT, 8, 1>(out, ring, splits, r0, rows, mt * LN_BM, nt * BN, N, tid - 64);
        }
        cluster_sync_all();                            // no CTA leaves while others read its partial
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) tc::tmem_dealloc(tm, 2 * BN);
    if (tid == 0 && sm.abort) atomicExch(&g_linear_error, (unsigned int)GDN_ERR_TIMEOUT);
}

// ------------------------------------------------------------------ launcher

constexpr size_t LN_SMEM = sizeof(LinearSmem) + 1024;
static_assert(LN_SMEM <= 232448, "one CTA per SM");
template <int BN> constexpr size_t pair_smem() { return sizeof(PairSmem<BN>) + 1024; }

static cudaLaunchConfig_t cluster_config(cudaLaunchAttribute (&attr)[2], int grid, int threads, size_t smem, int cluster,
                                         cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cfg;
}

// Set-up once per device: shared-memory attributes, and how many clusters can be
// resident at once.
struct LinearDevice {
    int split_clusters[9];                // of 2 to 8 CTAs of linear_kernel
    int pairs;                            // of pair_kernel
};

template <typename F> static bool max_clusters(F kernel, int threads, size_t smem, int cluster, int *n)
{
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = cluster_config(attr, cluster, threads, smem, cluster, nullptr);
    if (cudaOccupancyMaxActiveClusters(n, kernel, &cfg) == cudaSuccess) return true;
    cudaGetLastError();                                // a refused query
    *n = 0;
    return false;
}

template <typename TO, int ACT> static bool linear_attributes()
{
    const cudaFuncAttribute at = cudaFuncAttributeMaxDynamicSharedMemorySize;
    return cudaFuncSetAttribute(linear_kernel<TO, ACT>, at, (int)LN_SMEM) == cudaSuccess &&
           cudaFuncSetAttribute(pair_kernel<TO, 128, ACT>, at, (int)pair_smem<128>()) == cudaSuccess &&
           cudaFuncSetAttribute(pair_kernel<TO, 256, ACT>, at, (int)pair_smem<256>()) == cudaSuccess;
}

static const LinearDevice *linear_device()
{
    static LinearDevice info[64];
    static bool ready[64] = {};
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
    std::lock_guard<std::mutex> lock(mu);
    if (!ready[dev]) {
        if (!linear_attributes<float, 0>() || !linear_attributes<float, 1>() || !linear_attributes<float, 2>() ||
            !linear_attributes<float, 3>() || !linear_attributes<bf16, 0>() || !linear_attributes<bf16, 1>() ||
            !linear_attributes<bf16, 2>() || !linear_attributes<bf16, 3>())
            return nullptr;
        for (int k = 2; k <= 8; ++k)
            max_clusters(linear_kernel<bf16, 0>, LN_THREADS, LN_SMEM, k, &info[dev].split_clusters[k]);
        if (!max_clusters(pair_kernel<bf16, 256, 0>, PR_THREADS, pair_smem<256>(), 2, &info[dev].pairs) || info[dev].pairs < 1)
            return nullptr;
        ready[dev] = true;
    }
    return &info[dev];
}

struct LinearCall {
    const void *x, *w;
    long long x_row;
    int M, N, K;
    LinearOut out;
    cudaStream_t s;
};

template <typename TO, int BN, int ACT>
static cudaError_t launch_pairs(const LinearCall &c, const LinearDevice &dev)
{
    CUtensorMap mx, mw;
    if (!make_bf16_strided_map(&mx, c.x, c.M, c.K, c.x_row, LN_BM) || !make_bf16_strided_map(&mw, c.w, c.N, c.K, c.K, BN / 2))
        return cudaErrorInvalidValue;
    const int tiles = ((c.M + 255) / 256) * ((c.N + BN - 1) / BN);
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg =
        cluster_config(attr, 2 * (tiles < dev.pairs ? tiles : dev.pairs), PR_THREADS, pair_smem<BN>(), 2, c.s);
    return cudaLaunchKernelEx(&cfg, pair_kernel<TO, BN, ACT>, mx, mw, c.out, c.M, c.N, c.K);
}

template <typename TO, int ACT>
static cudaError_t launch_split(const LinearCall &c, const LinearDevice &dev, int n_sm)
{
    CUtensorMap mx, mw;
    const int a_rows = c.M < LN_BM ? (c.M + 7) & ~7 : LN_BM;
    const int fit = (int)((LN_RING - LN_A_BYTES) / (2 * ((uint32_t)a_rows * LN_BK * 2 + LN_B_BYTES))), stages = fit < LN_MAX_STAGES ? fit : LN_MAX_STAGES;
    if (!make_bf16_strided_map(&mx, c.x, c.M, c.K, c.x_row, a_rows) || !make_bf16_strided_map(&mw, c.w, c.N, c.K, c.K, LN_BN))
        return cudaErrorInvalidValue;
    const int n_work = ((c.M + LN_BM - 1) / LN_BM) * ((c.N + 127) / 128), kb_all = (c.K + LN_BK - 1) / LN_BK;
    // split K as far as the SMs reach, every CTA has a slice, and all clusters of that
    // size can be resident at once
    int splits = 8;
    while (splits > 1 && ((long long)n_work * splits > n_sm || splits > kb_all || dev.split_clusters[splits] < n_work)) --splits;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = cluster_config(attr, splits > 1 ? n_work * splits : (n_work < n_sm ? n_work : n_sm),
                                                  LN_THREADS, LN_SMEM, splits, c.s);
    return cudaLaunchKernelEx(&cfg, linear_kernel<TO, ACT>, mx, mw, c.out, c.M, c.N, c.K, splits, a_rows, stages);
}

// The form. Tiles of 256 columns once they are more than half of what the pairs hold, else of 128, which
// then fit one wave: 768 x 2,048 x 4,096 24.3 us with 256 and 19.8 with 128, 1,536 x 2,048 x 4,096 25.1 and
// 35.2. Split K by lone CTAs up to half of that wave: 256 x 2,048 x 4,096 12.0 us; from there
// to the whole wave it is within 10% either way (384 rows 14.5 in both, 1,024 18.2 here against 20.0).
template <typename TO, int ACT>
static cudaError_t launch_act(const LinearCall &c, const LinearDevice &dev, int n_sm)
{
    const long long m2 = (c.M + 255) / 256, t256 = m2 * ((c.N + 255) / 256), t128 = m2 * ((c.N + 127) / 128);
    if (c.M <= 128 || 2 * t128 <= dev.pairs) return launch_split<TO, ACT>(c, dev, n_sm);
    return 2 * t256 > dev.pairs ? launch_pairs<TO, 256, ACT>(c, dev) : launch_pairs<TO, 128, ACT>(c, dev);
}

template <typename TO>
static cudaError_t launch_out(const LinearCall &c, const LinearDevice &dev, int n_sm, gdn_activation act)
{
    switch (act) {
        case GDN_ACT_SILU: return launch_act<TO, GDN_ACT_SILU>(c, dev, n_sm);
        case GDN_ACT_GELU: return launch_act<TO, GDN_ACT_GELU>(c, dev, n_sm);
        case GDN_ACT_SIGMOID: return launch_act<TO, GDN_ACT_SIGMOID>(c, dev, n_sm);
        default: return launch_act<TO, GDN_ACT_NONE>(c, dev, n_sm);
    }
}

cudaError_t launch_linear(const void *x, long long x_row, const void *w, const float *bias, const void *residual,
                          long long r_row, void *y, long long y_row, int M, int N, int K, gdn_activation act,
                          gdn_dtype out_dt, cudaStream_t s)
{
    const int n_sm = sm_count();
    const LinearDevice *dev = linear_device();
    if (n_sm <= 0 || !dev) return cudaErrorInvalidDevice;
    const LinearCall c = {x, w, x_row, M, N, K, {bias, residual, y, r_row, y_row}, s};
    return out_dt == GDN_F32 ? launch_out<float>(c, *dev, n_sm, act) : launch_out<bf16>(c, *dev, n_sm, act);
}

// Device address of this file's error word, for gdn_device_error (NULL if the lookup fails).
void *linear_error_word()
{
    void *p = nullptr;
    return cudaGetSymbolAddress(&p, g_linear_error) == cudaSuccess ? p : nullptr;
}

}  // namespace gdn
