// gdn_norm.cu -- between two blocks of a layer ("qwen35moe -- Forward-Pass Design
// (Pantheon port)", the block scaffold: residual, then the next block's RMSNorm):
//   x' = x + res_scale * gate * n(delta),   n(d) = d (mean d^2 + eps)^-1/2 post_w, or d
//   h  = x' (mean x'^2 + eps)^-1/2 norm_w
// in one pass over a row of 2048. The sum x' is normed unrounded, in fp32.
//
// A CTA of 256 threads takes one row, 8 consecutive elements a thread, so that
// every access is a 16- or 32-byte vector of a dense row and a row's squares meet in
// one barrier. 4,096 rows with an fp32 stream, a post-norm and gates: 20.7 us, 5.7 TB/s of
// the copy's 6.8 (four CTAs per SM, as registers allow unasked: 21.6); with a bf16 stream and neither
// 11.9 us, 5.6 TB/s; one row: 2 us, latency.
#include "gdn_layer.cuh"

namespace gdn {

constexpr int NORM_THREADS = LD / 8;

struct NormArgs {
    const void *x, *delta, *gate;
    void *x_out, *h;
    const float *norm_w, *post_w;
    long long x_row, delta_row, gate_row, x_out_row, h_row;
    float res_scale, eps;
    int M;
};

// Sum over the CTA's 8 warps; `part` is used once per call.
__device__ __forceinline__ float row_sum(float v, float *part, int warp, int lane)
{
    v = warp_sum(v);
    if (lane == 0) part[warp] = v;
    __syncthreads();
    const float4 a = reinterpret_cast<const float4 *>(part)[0], b = reinterpret_cast<const float4 *>(part)[1];
    return ((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w));
}

// v * (mean v^2 + eps)^-1/2 over the row. Rows whose squares leave fp32 (or lose
// their bits below it, where eps does not cover that) are scaled by 2^-+100 first;
// the whole CTA sees the same sum, so the choice is uniform.
__device__ __forceinline__ void row_norm(float (&v)[8], float eps, float (*part)[8], int warp, int lane)
{
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(v[i], v[i], s);
    float ms = row_sum(s, part[0], warp, lane) * (1.0f / LD) + eps;
    if (!(ms > 1e-30f && ms < 1e36f)) {
        const float f = ms < 1.0f ? 0x1p100f : 0x1p-100f;          // NaN: either
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] *= f;
            s = fmaf(v[i], v[i], s);
        }
        ms = row_sum(s, part[1], warp, lane) * (1.0f / LD) + eps * f * f;
    }
    const float r = 1.0f / sqrtf(ms);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= r;
}

template <typename TS, typename TA, bool GATE, bool POST>
__global__ void __launch_bounds__(NORM_THREADS, 5) add_norm_kernel(const NormArgs a)
{
    __shared__ __align__(16) float part[4][8];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, c = tid * 8;
    const size_t m = blockIdx.x;
    grid_dep_wait();
    grid_dep_launch();
    float x[8], d[8], g[8], w[8];
    ld8(static_cast<const TS *>(a.x) + m * a.x_row + c, x);
    const bool add = a.delta != nullptr;
    if (add) ld8(static_cast<const TA *>(a.delta) + m * a.delta_row + c, d);
    if (GATE) ld8(static_cast<const TA *>(a.gate) + m * a.gate_row + c, g);
    if (a.h) ld8(a.norm_w + c, w);
    if (add) {
        if (POST) {
            float pw[8];
            ld8(a.post_w + c, pw);
            row_norm(d, a.eps, part, warp, lane);
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] *= pw[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = fmaf(a.res_scale, GATE ? d[i] * g[i] : d[i], x[i]);
    }
    if (a.x_out) st8(static_cast<TS *>(a.x_out) + m * a.x_out_row + c, x);
    if (a.h) {
        row_norm(x, a.eps, part + 2, warp, lane);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= w[i];
        st8(static_cast<TA *>(a.h) + m * a.h_row + c, x);
    }
}

template <typename TS, typename TA>
static cudaError_t launch_t(const NormArgs &a, cudaStream_t s)
{
    const dim3 g(a.M), b(NORM_THREADS);
    if (a.gate)
        return a.post_w ? launch_pdl(add_norm_kernel<TS, TA, true, true>, g, b, 0, s, a)
                        : launch_pdl(add_norm_kernel<TS, TA, true, false>, g, b, 0, s, a);
    return a.post_w ? launch_pdl(add_norm_kernel<TS, TA, false, true>, g, b, 0, s, a)
                    : launch_pdl(add_norm_kernel<TS, TA, false, false>, g, b, 0, s, a);
}

cudaError_t launch_add_norm(const gdn_norm_params *p, const void *x, long long x_row, const void *delta,
                            long long delta_row, const void *gate, long long gate_row, void *x_out,
                            long long x_out_row, void *h, long long h_row, int M, gdn_dtype stream_dt, gdn_dtype act,
                            cudaStream_t s)
{
    const NormArgs a = {x, delta, gate, x_out, h, p->norm_w, p->post_w, x_row, delta_row, gate_row, x_out_row, h_row,
                        p->res_scale, p->norm_eps, M};
    if (stream_dt == GDN_F32) return act == GDN_F32 ? launch_t<float, float>(a, s) : launch_t<float, bf16>(a, s);
    return act == GDN_F32 ? launch_t<bf16, float>(a, s) : launch_t<bf16, bf16>(a, s);
}

}  // namespace gdn
