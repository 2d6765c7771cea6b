// gdn_linear.cu -- y = residual + act(x w^T + bias) on 5th-generation tensor cores:
// bf16 operands, fp32 accumulation, everything behind the product in the
// epilogue, on the fp32 accumulators, with one rounding at the end. The dense
// products of "qwen35moe -- Forward-Pass Design (Pantheon port)" that have no
// entry point of their own: steps 1 and 7 of section "Full-attention block"
// (joint query and gate, key and value projection; attn_output with the residual).
//
// Tiles of 128 rows x BN columns (BN = 256, or 128 where the 256-wide tiles fill
// at most half of the SMs) over a persistent grid: a TMA warp, an MMA warp, four epilogue
// warps with the accumulators double-buffered in tensor memory. Where the tiles are
// too few for the GPU, each tile's K range is split over the CTAs of a cluster,
// whose partial tiles meet in distributed shared memory (always in the same order).
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
    int act;
};

__device__ __forceinline__ float apply_act(float v, int act)
{
    if (act == GDN_ACT_SILU) return v / (1.0f + __expf(-v));
    if (act == GDN_ACT_GELU) return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
    if (act == GDN_ACT_SIGMOID) return 1.0f / (1.0f + __expf(-v));
    return v;
}

// Epilogue of 8 neighbouring columns of row m.
template <typename TO>
__device__ __forceinline__ void finish8(const LinearOut &o, int m, int n, float (&v)[8])
{
    if (o.bias) {
        float b[8];
        ld8(o.bias + n, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += b[i];
    }
    if (o.act != GDN_ACT_NONE) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = apply_act(v[i], o.act);
    }
    if (o.residual) {
        float r[8];
        ld8(static_cast<const TO *>(o.residual) + (size_t)m * o.r_row + n, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += r[i];
    }
    st8(static_cast<TO *>(o.y) + (size_t)m * o.y_row + n, v);
}

template <int BN>
struct LinearSmem {
    static constexpr int STAGES = BN == 256 ? 4 : 6;
    static constexpr uint32_t STAGE_BYTES = LN_A_BYTES + BN * LN_BK * 2;
    static constexpr int PART_LD = BN + 4;
    static_assert(LN_BM * PART_LD * 4 <= STAGES * STAGE_BYTES, "a partial tile fits the stages");
    alignas(1024) unsigned char stage[STAGES][STAGE_BYTES];
    alignas(8) uint64_t full[STAGES], empty[STAGES], acc_full[2], acc_empty[2];
    int last_it[STAGES];
    uint32_t tmem;
    int abort;
};

template <typename TO, int BN>
__global__ void __launch_bounds__(LN_THREADS, 1)
    linear_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw, const LinearOut out,
                  int M, int N, int K, int splits)
{
    using Smem = LinearSmem<BN>;
    constexpr int STAGES = Smem::STAGES, PLD = Smem::PART_LD;
    extern __shared__ unsigned char smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
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
    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&sm.full[s]), 1);
            mbar_init(smem_u32(&sm.empty[s]), 1);
            sm.last_it[s] = -1;
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
            int it = 0;
            for (int w = w0; w < wend && !aborted; w += wstep) {
                const int mt = w / n_tiles, nt = w % n_tiles;
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    const int s = it % STAGES;
                    if (it >= STAGES && !mbar_wait_bounded(smem_u32(&sm.empty[s]), (uint32_t)((it / STAGES - 1) & 1)))
                        sm.abort = 1;
                    if (aborted) break;
                    const uint32_t dst = smem_u32(sm.stage[s]), bar = smem_u32(&sm.full[s]);
                    mbar_arrive_expect_tx(bar, Smem::STAGE_BYTES);
                    tma_load_2d(dst, &mx, kb * LN_BK, mt * LN_BM, bar);
                    tma_load_2d(dst + LN_A_BYTES, &mw, kb * LN_BK, nt * BN, bar);
                    sm.last_it[s] = it;
                }
            }
            if (aborted)                               // copies in flight land before the CTA exits
                for (int s = 0; s < STAGES; ++s)
                    if (sm.last_it[s] >= 0)
                        mbar_wait_bounded(smem_u32(&sm.full[s]), (uint32_t)((sm.last_it[s] / STAGES) & 1));
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = tc::instr_desc(tc::FMT_BF16, LN_BM, BN);
            int it = 0, ti = 0;
            for (int w = w0; w < wend && !aborted; w += wstep, ++ti) {
                const int ab = ti & 1;
                if (ti >= 2 && !mbar_wait_bounded(smem_u32(&sm.acc_empty[ab]), (uint32_t)(((ti >> 1) - 1) & 1)))
                    sm.abort = 1;
                tc::fence_after_sync();
                const uint32_t d = tm + (uint32_t)(BN * ab);
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    const int s = it % STAGES;
                    if (!mbar_wait_bounded(smem_u32(&sm.full[s]), (uint32_t)((it / STAGES) & 1))) sm.abort = 1;
                    if (aborted) break;
                    tc::fence_after_sync();
                    const uint64_t ad = tc::sw128_desc(smem_u32(sm.stage[s]));
                    const uint64_t bd = tc::sw128_desc(smem_u32(sm.stage[s]) + LN_A_BYTES);
#pragma unroll
                    for (int k = 0; k < LN_BK / 16; ++k)
                        tc::mma_f16(d, ad + 2u * k, bd + 2u * k, idesc, (kb > kb0 || k > 0) ? 1u : 0u);
                    tc::mma_commit(smem_u32(&sm.empty[s]));
                }
                if (aborted) break;
                tc::mma_commit(smem_u32(&sm.acc_full[ab]));
            }
        }
    } else {
        const int q = warp & 3, row = 32 * q + lane;
        if (split) {                                   // this CTA's fp32 partial tile into shared memory
            if (!mbar_wait_bounded(smem_u32(&sm.acc_full[0]), 0)) sm.abort = 1;
            tc::fence_after_sync();
            float *p = reinterpret_cast<float *>(sm.stage[0]) + row * PLD;
            for (int c = 0; c < BN; c += 32) {
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
            if (aborted) break;
            tc::fence_after_sync();
            const int m = mt * LN_BM + row;
            for (int c = 0; c < BN; c += 32) {
                float v[32];
                tc::tmem_ld32(tc::tmem_addr(tm + (uint32_t)(BN * ab), 32 * q, c), v);
                tc::wait_ld();
                const int n = nt * BN + c;
                if (m < M) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (n + 8 * e < N) finish8<TO>(out, m, n + 8 * e, *reinterpret_cast<float(*)[8]>(v + 8 * e));
                }
            }
            tc::fence_before_sync();
            mbar_arrive(smem_u32(&sm.acc_empty[ab]));
        }
    }
    if (split) {
        // CTA r of the cluster writes rows [r 128/S, (r+1) 128/S) of the tile, each the sum of the S partials
        cluster_sync_all();
        if (warp >= 2 && !aborted) {
            const int rows = LN_BM / splits, r0 = part * rows;
            const int mt = w0 / n_tiles, nt = w0 % n_tiles;
            const uint32_t base = smem_u32(sm.stage[0]);
            for (int f = tid - 64; f < rows * (BN / 8); f += 128) {
                const int rr = r0 + f / (BN / 8), col = 8 * (f % (BN / 8));
                const int m = mt * LN_BM + rr, n = nt * BN + col;
                if (m >= M || n >= N) continue;
                const uint32_t off = base + (uint32_t)((rr * PLD + col) * 4);
                float4 a[8], b[8];                     // all remote loads in flight before the sum
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (r < splits) {
                        const uint32_t at = mapa_shared(off, (uint32_t)r);
                        a[r] = ld_cluster_f32x4(at);
                        b[r] = ld_cluster_f32x4(at + 16);
                    }
                float v[8] = {a[0].x, a[0].y, a[0].z, a[0].w, b[0].x, b[0].y, b[0].z, b[0].w};
#pragma unroll
                for (int r = 1; r < 8; ++r)
                    if (r < splits) {
                        v[0] += a[r].x; v[1] += a[r].y; v[2] += a[r].z; v[3] += a[r].w;
                        v[4] += b[r].x; v[5] += b[r].y; v[6] += b[r].z; v[7] += b[r].w;
                    }
                finish8<TO>(out, m, n, v);
            }
        }
        cluster_sync_all();                            // no CTA leaves while others read its partial
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) tc::tmem_dealloc(tm, 2 * BN);
    if (tid == 0 && sm.abort) atomicExch(&g_linear_error, (unsigned int)GDN_ERR_TIMEOUT);
}

// ------------------------------------------------------------------ launcher

template <int BN>
constexpr size_t linear_smem() { return sizeof(LinearSmem<BN>) + 1024; }

// Set-up once per device: shared-memory attributes, and how many clusters of 2,
// 4 and 8 CTAs can be resident at once.
struct LinearDevice {
    int max_clusters[2][3];   // [BN == 128]
};

template <int BN>
static bool linear_setup(int (&max_clusters)[3])
{
    if (cudaFuncSetAttribute(linear_kernel<float, BN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)linear_smem<BN>()) != cudaSuccess ||
        cudaFuncSetAttribute(linear_kernel<bf16, BN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)linear_smem<BN>()) != cudaSuccess)
        return false;
    for (int k = 0; k < 3; ++k) {
        cudaLaunchConfig_t q = {};
        q.gridDim = dim3(2 << k);
        q.blockDim = dim3(LN_THREADS);
        q.dynamicSmemBytes = linear_smem<BN>();
        cudaLaunchAttribute qa[1];
        qa[0].id = cudaLaunchAttributeClusterDimension;
        qa[0].val.clusterDim.x = 2u << k;
        qa[0].val.clusterDim.y = 1;
        qa[0].val.clusterDim.z = 1;
        q.attrs = qa;
        q.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, linear_kernel<bf16, BN>, &q) != cudaSuccess) {
            cudaGetLastError();                        // a refused query: never split this far
            n = 0;
        }
        max_clusters[k] = n;
    }
    return true;
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
        if (!linear_setup<256>(info[dev].max_clusters[0]) || !linear_setup<128>(info[dev].max_clusters[1])) return nullptr;
        ready[dev] = true;
    }
    return &info[dev];
}

template <int BN>
static cudaError_t launch_bn(const void *x, long long x_row, const void *w, const LinearOut &out, int M, int N, int K,
                             gdn_dtype out_dt, cudaStream_t s, int n_sm, const int (&max_clusters)[3])
{
    CUtensorMap mx, mw;
    if (!make_bf16_strided_map(&mx, x, M, K, x_row, LN_BM) || !make_bf16_strided_map(&mw, w, N, K, K, BN))
        return cudaErrorInvalidValue;
    const int n_work = ((M + LN_BM - 1) / LN_BM) * ((N + BN - 1) / BN), kb_all = (K + LN_BK - 1) / LN_BK;
    // split K while the tiles fill at most half of the SMs, and only as far as all
    // clusters of that size can be resident at once
    int splits = 1;
    while (splits < 8 && n_work * splits * 2 <= n_sm && splits * 2 <= kb_all &&
           max_clusters[splits == 1 ? 0 : splits == 2 ? 1 : 2] >= n_work)
        splits *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(splits > 1 ? n_work * splits : (n_work < n_sm ? n_work : n_sm));
    cfg.blockDim = dim3(LN_THREADS);
    cfg.dynamicSmemBytes = linear_smem<BN>();
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)splits;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = splits > 1 ? 2 : 1;
    return out_dt == GDN_F32 ? cudaLaunchKernelEx(&cfg, linear_kernel<float, BN>, mx, mw, out, M, N, K, splits)
                             : cudaLaunchKernelEx(&cfg, linear_kernel<bf16, BN>, mx, mw, out, M, N, K, splits);
}

cudaError_t launch_linear(const void *x, long long x_row, const void *w, const float *bias, const void *residual,
                          long long r_row, void *y, long long y_row, int M, int N, int K, gdn_activation act,
                          gdn_dtype out_dt, cudaStream_t s)
{
    const int n_sm = sm_count();
    const LinearDevice *dev = linear_device();
    if (n_sm <= 0 || !dev) return cudaErrorInvalidDevice;
    const LinearOut o = {bias, residual, y, r_row, y_row, (int)act};
    if ((long long)((M + LN_BM - 1) / LN_BM) * ((N + 255) / 256) * 2 <= n_sm)
        return launch_bn<128>(x, x_row, w, o, M, N, K, out_dt, s, n_sm, dev->max_clusters[1]);
    return launch_bn<256>(x, x_row, w, o, M, N, K, out_dt, s, n_sm, dev->max_clusters[0]);
}

// Device address of this file's error word, for gdn_device_error (NULL if the lookup fails).
void *linear_error_word()
{
    void *p = nullptr;
    return cudaGetSymbolAddress(&p, g_linear_error) == cudaSuccess ? p : nullptr;
}

}  // namespace gdn
