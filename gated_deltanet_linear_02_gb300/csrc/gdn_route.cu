// gdn_route.cu -- the router of the mixture-of-experts feed-forward ("qwen35moe --
// Forward-Pass Design (Pantheon port)", the MoE section): logits x . router^T of E
// experts, the top_k of them per token, and softmax weights.
//
// A cluster of S CTAs takes 128 tokens, CTA r the r-th part of K = 2048: all E logits
// of a token come from one tcgen05 product (M = 128 tokens, N = E), with K split so
// that few tokens still spread over SMs. Every 256 of K have an accumulator of
// their own; those partial sums are added in fp32 rounded to nearest (the tensor
// core truncates its sums, so short ones keep the logits' error near 1e-7 of their
// terms). They meet in distributed shared memory, where each CTA has 128 / S
// tokens: a warp per token holds 8 logits a lane and takes the largest k times.
//
// The choice is exact: where two of the first k + 1 logits are closer than a bound on their
// error, the warp sums theirs again in pairs of fp32 (48 bits; products of bf16 are exact).
// The bound: an accumulator takes 16 steps, each off by at most 2^-23 of its sum of magnitudes,
// and up to 8 roundings of 2^-24 join them: 1.25 2^-19 of sum |x_i r_i| in all, twice that for a
// difference. That sum is at most |x| |r| in each part of K; warps that the products leave
// idle take the norms from the stages as they pass (of r the largest).
// Ties go to the lowest index. NaN ranks below everything. 256 tokens 17.9 us, 4,096
// 22.9 us, 4 tokens 8.2: the products are done after 1.7 us, the partial logits of a CTA's
// tokens take 5 (131 KB from the other SMs), the choice 2, near ties 4, the bound's norms 1.
//
// Where a wait of a cluster gave up, its tokens are marked as nobody's (id -1), so that the kernels
// behind find no index that was not written. `lose` makes that happen, for the library's self-test:
// the products' completion is not announced, and every wait for it runs out.
#include <mutex>

#include "gdn_layer.cuh"
#include "gdn_moe.cuh"
#include "gdn_route.cuh"
#include "gdn_tc.cuh"
#include "gdn_tma.cuh"

namespace gdn {

__device__ unsigned int g_route_error;    // GDN_ERR_TIMEOUT if a bounded wait gave up

__device__ __forceinline__ int ld_cluster_s32(uint32_t addr)
{
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

constexpr int RT_BM = MOE_ROUTE_TILE, RT_BK = 64, RT_THREADS = 512, RT_STAGES = 4;
constexpr uint32_t RT_A_BYTES = RT_BM * RT_BK * 2;
constexpr int RT_ACC_K = 256;             // K of one accumulator

struct RouteSmem {
    alignas(1024) unsigned char stage[RT_STAGES][RT_A_BYTES + RT_MAX_E * RT_BK * 2];
    alignas(8) uint64_t full[RT_STAGES], empty[RT_STAGES], done;
    int last_it[RT_STAGES];
    float x_squares[RT_BM];               // sums of squares of this part of the tokens' rows
    uint32_t row_norm;                    // bits of the largest norm of this part of the router's rows
    uint32_t tmem;
    int abort;
};
constexpr int RT_NORM_WARP = 8, RT_NORM_WARPS = 8;       // a thread per router row
static_assert(32 * RT_NORM_WARPS == RT_MAX_E && 32 * (RT_NORM_WARP + RT_NORM_WARPS) == RT_THREADS, "a thread per router row");

// The norm of n bf16 values from their sum of squares; where that left fp32's range, a bound on it
// from the largest magnitude (bits `top`). 0 if a value is not finite: then so is the
// logit, and there is nothing to settle.
__device__ __forceinline__ bool in_range(float squares) { return squares > 0x1p-80f && squares < 0x1p100f; }
__device__ __forceinline__ float norm_of(float squares, uint32_t top, int n)
{
    if (in_range(squares)) return sqrtf(squares);
    return top >= 0x7f80u ? 0.0f : sqrtf((float)n) * __uint_as_float(top << 16);
}
// The sum of squares of 8 values, to 1 in 128: four products and sums of pairs in bf16, then fp32.
__device__ __forceinline__ float squares(uint4 u)
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t t;
    asm("mul.rn.bf16x2 %0, %1, %1;" : "=r"(t) : "r"(w[0]));
#pragma unroll
    for (int i = 1; i < 4; ++i) asm("fma.rn.bf16x2 %0, %1, %1, %0;" : "+r"(t) : "r"(w[i]));
    return __uint_as_float(t << 16) + __uint_as_float(t & 0xFFFF0000u);
}
__device__ __forceinline__ uint32_t top_bits(uint4 u)
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) t = max(t, max(w[i] & 0x7fffu, w[i] >> 16 & 0x7fffu));
    return t;
}

// The bound where the squares of part of a row left fp32's range (zeros too): by the whole row, in memory.
static __device__ __noinline__ float bound_of(const bf16 *x, float r_norm, int splits, int lane)
{
    float q = 0.0f;
    uint32_t top = 0;
    for (int c = 0; c < LD; c += 256) {
        const uint4 u = *reinterpret_cast<const uint4 *>(x + c + lane * 8);
        q += squares(u);
        top = max(top, top_bits(u));
    }
    const float norm = norm_of(warp_sum(q), __reduce_max_sync(0xffffffffu, top), LD);
    return norm == 0.0f ? 0.0f : norm * sqrtf((float)splits) * __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(r_norm)));
}
constexpr float RT_TIE = 0x1.5p-18f;      // 1.25 2^-18 and what the norms' own roundings take

static_assert(RT_BM * (RT_MAX_E + 4) * 4 <= sizeof(RouteSmem::stage), "partial logits fit the stages");

__global__ void __launch_bounds__(RT_THREADS, 1)
    route_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mr, const bf16 *x,
                 long long x_row, const bf16 *router, int M, int E, int N, int k, int renorm, int splits,
                 int32_t *ids, float *weights, MoePlaces places, int *state, int n_state, int lose)
{
    extern __shared__ unsigned char smem_raw[];
    RouteSmem &sm = *reinterpret_cast<RouteSmem *>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tile = (int)blockIdx.x / splits, part = (int)blockIdx.x % splits;
    const int kbn = LD / RT_BK / splits, kb0 = part * kbn;                 // 4 to 16 K slices
    const int naccs = (kbn * RT_BK + RT_ACC_K - 1) / RT_ACC_K;             // 1 or 2 (splits >= 4)
    const int PLD = N + 4;
    const uint32_t cols = naccs > 1 ? 512u : 256u;
    const volatile int &aborted = sm.abort;

    if (warp == 1) {
        tc::tmem_alloc(smem_u32(&sm.tmem), cols);
        tc::tmem_relinquish();
    }
    if (tid == 0) {
        for (int s = 0; s < RT_STAGES; ++s) {
            mbar_init(smem_u32(&sm.full[s]), 1);
            mbar_init(smem_u32(&sm.empty[s]), 1 + RT_NORM_WARPS);
            sm.last_it[s] = -1;
        }
        mbar_init(smem_u32(&sm.done), 1);
        sm.row_norm = 0u;
        sm.abort = 0;
        fence_mbar_init();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = sm.tmem;
    grid_dep_wait();
    grid_dep_launch();
    // with a single cluster the counters that the choice adds to are cleared here: the barrier
    // before the choice orders it
    if (part == 0)
        for (int i = tid; i < n_state; i += RT_THREADS) state[i] = 0;

    if (warp == 0) {
        if (lane == 0) {
            for (int it = 0; it < kbn; ++it) {
                const int s = it % RT_STAGES;
                if (it >= RT_STAGES && !mbar_wait_bounded(smem_u32(&sm.empty[s]), (uint32_t)((it / RT_STAGES - 1) & 1)))
                    sm.abort = 1;
                if (aborted) break;
                const uint32_t dst = smem_u32(sm.stage[s]), bar = smem_u32(&sm.full[s]);
                mbar_arrive_expect_tx(bar, RT_A_BYTES + (uint32_t)N * RT_BK * 2);
                tma_load_2d(dst, &mx, (kb0 + it) * RT_BK, tile * RT_BM, bar);
                tma_load_2d(dst + RT_A_BYTES, &mr, (kb0 + it) * RT_BK, 0, bar);
                sm.last_it[s] = it;
            }
            if (aborted)
                for (int s = 0; s < RT_STAGES; ++s)
                    if (sm.last_it[s] >= 0)
                        mbar_wait_bounded(smem_u32(&sm.full[s]), (uint32_t)((sm.last_it[s] / RT_STAGES) & 1));
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = tc::instr_desc(tc::FMT_BF16, RT_BM, N);
            for (int it = 0; it < kbn; ++it) {
                const int s = it % RT_STAGES;
                if (!mbar_wait_bounded(smem_u32(&sm.full[s]), (uint32_t)((it / RT_STAGES) & 1))) sm.abort = 1;
                if (aborted) break;
                tc::fence_after_sync();
                const uint64_t ad = tc::sw128_desc(smem_u32(sm.stage[s]));
                const uint64_t bd = tc::sw128_desc(smem_u32(sm.stage[s]) + RT_A_BYTES);
                const int in = it % (RT_ACC_K / RT_BK);
                const uint32_t d = tm + 256u * (uint32_t)(it / (RT_ACC_K / RT_BK));
#pragma unroll
                for (int kk = 0; kk < RT_BK / 16; ++kk)
                    tc::mma_f16(d, ad + 2u * kk, bd + 2u * kk, idesc, (in > 0 || kk > 0) ? 1u : 0u);
                tc::mma_commit(smem_u32(&sm.empty[s]));
            }
            if (!aborted && !lose) tc::mma_commit(smem_u32(&sm.done));
        }
    } else if (warp >= 4 && warp < 8) {
        if (!mbar_wait_bounded(smem_u32(&sm.done), 0)) sm.abort = 1;
        const bool lost = warp_gave_up(aborted);
        asm volatile("bar.sync 1, %0;" ::"n"(128 + 32 * RT_NORM_WARPS) : "memory");       // the norms are done with the stages
        tc::fence_after_sync();
        const int q = warp & 3, row = 32 * q + lane;
        float *p = reinterpret_cast<float *>(sm.stage[0]) + row * PLD;
        if (!lost)
            for (int c = 0; c < N; c += 16) {
                float v[16];
                tc::tmem_ld16(tc::tmem_addr(tm, 32 * q, c), v);
                if (naccs > 1) {
                    float u[16];
                    tc::tmem_ld16(tc::tmem_addr(tm, 32 * q, 256 + c), u);
                    tc::wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] += u[i];
                } else {
                    tc::wait_ld();
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    reinterpret_cast<float4 *>(p + c)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            }
    }
    const int rows = RT_BM / splits;
    if (warp >= RT_NORM_WARP) {
        const int e = tid - 32 * RT_NORM_WARP;
        const int row = e >> 1, half = (e & 1) << 2;   // of x: half a row a thread
        float q = 0.0f, qx = 0.0f;
        for (int it = 0; it < kbn; ++it) {
            const int s = it % RT_STAGES;
            if (!mbar_wait_sleep(smem_u32(&sm.full[s]), (uint32_t)((it / RT_STAGES) & 1))) sm.abort = 1;
            if (warp_gave_up(aborted)) break;
            // 16 bytes at a time, in an order that keeps the lanes off each other's banks
            const unsigned char *r = sm.stage[s] + RT_A_BYTES + e * (RT_BK * 2), *rx = sm.stage[s] + row * (RT_BK * 2);
            if (e < E)
#pragma unroll
                for (int j = 0; j < 8; ++j) q += squares(*reinterpret_cast<const uint4 *>(r + ((j ^ (e & 7)) << 4)));
#pragma unroll
            for (int j = 0; j < 4; ++j) qx += squares(*reinterpret_cast<const uint4 *>(rx + (((j | half) ^ (row & 7)) << 4)));
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.empty[s]));
        }
        __syncwarp();
        asm volatile("bar.arrive 1, %0;" ::"n"(128 + 32 * RT_NORM_WARPS) : "memory");
        qx += __shfl_xor_sync(0xffffffffu, qx, 1);
        if (half == 0) sm.x_squares[row] = qx;
        float norm = norm_of(q, 0u, 0);
        if (e < E && !(norm > 0.0f)) {                 // squares out of range
            uint32_t top = 0;
            for (int c = 0; c < kbn * RT_BK; c += 8)
                top = max(top, top_bits(*reinterpret_cast<const uint4 *>(router + (size_t)e * LD + kb0 * RT_BK + c)));
            norm = norm_of(0.0f, top, kbn * RT_BK);
        }
        const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(norm));
        if (lane == 0) atomicMax(&sm.row_norm, most);
    }
    cluster_sync_all();
    {
        const uint32_t base = smem_u32(sm.stage[0]);
        for (int t = part * rows + warp; t < (part + 1) * rows; t += RT_THREADS / 32) {
            const int m = tile * RT_BM + t;
            if (m >= M) break;
            // whether any CTA of the cluster has given up: its partial logits may not be there
            const uint32_t peer = (uint32_t)min(lane, splits - 1);
            const int lost = ld_cluster_s32(mapa_shared(smem_u32(&sm.abort), peer));
            const float r_norm = __int_as_float(ld_cluster_s32(mapa_shared(smem_u32(&sm.row_norm), peer)));
            const float x_sq = __int_as_float(ld_cluster_s32(mapa_shared(smem_u32(&sm.x_squares[t]), peer)));
            float v[RT_SLOTS];
#pragma unroll
            for (int j = 0; j < RT_SLOTS; ++j) v[j] = 0.0f;
            // all loads in flight, 16 bytes each (a quarter of the requests to the other SMs)
            const bool low = 4 * lane < N, high = 128 + 4 * lane < N;
            float4 p[8], u[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                p[r] = u[r] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                const uint32_t at = mapa_shared(base + (uint32_t)(t * PLD + 4 * lane) * 4u, (uint32_t)min(r, splits - 1));
                if (r < splits && low) p[r] = ld_cluster_f32x4(at);
                if (r < splits && high) u[r] = ld_cluster_f32x4(at + 512u);
            }
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                v[0] += p[r].x; v[1] += p[r].y; v[2] += p[r].z; v[3] += p[r].w;
                v[4] += u[r].x; v[5] += u[r].y; v[6] += u[r].z; v[7] += u[r].w;
            }
            if (__any_sync(0xffffffffu, lost)) {       // nobody's token: what follows must not take these for indices
                if (lane < k) {
                    ids[(size_t)m * k + lane] = -1;
                    weights[(size_t)m * k + lane] = 0.0f;
                    if (places.count) places.rank[(size_t)m * k + lane] = -1;
                }
                continue;
            }
            int id;
            float w;
            float bound = warp_sum(lane < splits ? sqrtf(x_sq) * r_norm : 0.0f);
            if (__any_sync(0xffffffffu, !in_range(x_sq))) bound = bound_of(x + (size_t)m * x_row, r_norm, splits, lane);
            choose(v, E, k, renorm != 0, RT_TIE * bound, x + (size_t)m * x_row, router, lane, id, w);
            if (lane < k) {
                ids[(size_t)m * k + lane] = id;
                weights[(size_t)m * k + lane] = w;
                if (places.count) place_pair(places, m, lane, id, k);
            }
        }
    }
    cluster_sync_all();                                // no CTA leaves while others read its partial logits
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) tc::tmem_dealloc(tm, cols);
    if (tid == 0 && sm.abort) atomicExch(&g_route_error, (unsigned int)GDN_ERR_TIMEOUT);
}

static bool route_setup()
{
    static bool ready[64] = {};
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    std::lock_guard<std::mutex> lock(mu);
    if (!ready[dev]) {
        if (cudaFuncSetAttribute(route_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)sizeof(RouteSmem) + 1024) != cudaSuccess)
            return false;
        ready[dev] = true;
    }
    return true;
}

cudaError_t launch_route(const gdn_moe_params *p, const void *x, long long x_row, int M, int32_t *ids, float *weights,
                         const MoePlaces &places, int *state, int n_state, bool lose, cudaStream_t s)
{
    if (!route_setup()) return cudaErrorInvalidDevice;
    const int E = p->num_experts, N = (E + 15) & ~15;
    CUtensorMap mx, mr;
    if (!make_bf16_strided_map(&mx, x, M, LD, x_row, RT_BM) || !make_bf16_strided_map(&mr, p->router, E, LD, LD, N))
        return cudaErrorInvalidValue;
    const int tiles = (M + RT_BM - 1) / RT_BM, splits = tiles <= 16 ? 8 : 4;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(tiles * splits);
    cfg.blockDim = dim3(RT_THREADS);
    cfg.dynamicSmemBytes = sizeof(RouteSmem) + 1024;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)splits;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, route_kernel, mx, mr, (const bf16 *)x, x_row, (const bf16 *)p->router, M, E, N,
                              p->top_k, p->norm_topk, splits, ids, weights, places,
                              state, n_state, (int)lose);
}

cudaError_t launch_route_only(const gdn_moe_params *p, const void *x, long long x_row, int M, int32_t *ids,
                              float *weights, cudaStream_t s)
{
    return launch_route(p, x, x_row, M, ids, weights, MoePlaces{}, nullptr, 0, false, s);
}

// Device address of this file's error word, for gdn_device_error (NULL if the lookup fails).
void *route_error_word()
{
    void *p = nullptr;
    return cudaGetSymbolAddress(&p, g_route_error) == cudaSuccess ? p : nullptr;
}

}  // namespace gdn
