// gdn_paged.cu -- causal attention of new tokens over the paged cache (bf16 or
// 4 bits), steps 5-6 of section "Full-attention block" of "qwen35moe --
// Forward-Pass Design (Pantheon port)".
//
// One warp per (token, query head): 8 dims per lane, one pass over the context
// with the running maximum and sum of the softmax.
#include "gdn_async.cuh"
#include "gdn_kv.cuh"

namespace gdn {

struct PagedArgs {
    PagedBatch b;
    const void *ck, *cv;
    const bf16 *q, *gate;
    long long gate_row, gate_head;
    void *out;
};

template <bool Q4>
__device__ __forceinline__ void load_row(const PagedArgs &a, int page, int head, int off, bool isv, int lane, float (&x)[8])
{
    if (page < 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0.0f;
        return;
    }
    if (!Q4) {
        const uint4 u = __ldg(reinterpret_cast<const uint4 *>(static_cast<const bf16 *>(isv ? a.cv : a.ck) +
                                                              row_bf16(a.b, page, head, off)) + lane);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16));
    } else {
        const unsigned char *rec = static_cast<const unsigned char *>(a.ck) + record_of(a.b, page, head, off);
        const int r = off & (REC_ROWS - 1), g = lane >> 3, c = lane & 7;
        const uint32_t w = *reinterpret_cast<const uint32_t *>(rec + (isv ? REC_V : 0u) + r * 128 + c * 16 + g * 4);
        const uint32_t sz = *reinterpret_cast<const uint32_t *>(rec + (isv ? REC_VSZ : REC_KSZ) + r * 16 + g * 4);
        const float s = __uint_as_float(sz << 16), z = __uint_as_float(sz & 0xFFFF0000u);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = fmaf(s, (float)((w >> (4 * i)) & 15u), z);
    }
}

template <typename TO, bool Q4>
__global__ void __launch_bounds__(256) attn_paged_kernel(const PagedArgs a)
{
    const int lane = threadIdx.x & 31;
    const long long item = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int m = (int)(item / KV_HQ), h = (int)(item % KV_HQ);
    grid_dep_wait();
    grid_dep_launch();
    if (m >= a.b.M) return;
    const TokenPlace at = token_place(a.b, m, lane);
    if (at.seq < 0) return;
    const int n = min(at.pos + 1, a.b.max_pages << a.b.page_log2);
    float q[8], acc[8], M = -INFINITY, l = 0.0f;
    const uint4 u = __ldg(reinterpret_cast<const uint4 *>(a.q + ((size_t)m * KV_HQ + h) * KV_D) + lane);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        q[i] = 0.0625f * __uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16));
        acc[i] = 0.0f;
    }
    for (int p = 0; p < n; ++p) {
        const int page = cache_page(a.b, at.seq, p), off = p & (a.b.page - 1);
        float k[8], v[8], s = 0.0f;
        load_row<Q4>(a, page, h / KV_G, off, false, lane, k);
        load_row<Q4>(a, page, h / KV_G, off, true, lane, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(q[i], k[i], s);
        s = warp_sum(s);
        const float Mn = fmaxf(M, s), f = expf(M - Mn), e = expf(s - Mn);
        M = Mn;
        l = l * f + e;
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = acc[i] * f + e * v[i];
    }
    const float inv = n > 0 ? 1.0f / l : 0.0f;
    TO *out = static_cast<TO *>(a.out) + ((size_t)m * KV_HQ + h) * KV_D + 8 * lane;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float o = acc[i] * inv;
        if (a.gate != nullptr) o /= 1.0f + expf(-to_f(a.gate[m * a.gate_row + h * a.gate_head + 8 * lane + i]));
        out[i] = from_f<TO>(o);
    }
}

size_t paged_workspace_bytes(const gdn_paged_batch *, const gdn_kv_cache *) { return 16; }

cudaError_t launch_attn_paged(const gdn_paged_batch *b, const gdn_kv_cache *c, const void *q, const void *gate,
                              long long gate_row, long long gate_head, void *out, void *, gdn_dtype out_dt,
                              cudaStream_t s)
{
    PagedArgs a = {paged_batch(*b, *c), c->k, c->v, (const bf16 *)q, (const bf16 *)gate, gate_row, gate_head, out};
    const dim3 grid((unsigned)(((long long)b->M * KV_HQ + 7) / 8)), block(256);
    if (c->format == GDN_KV_Q4)
        return out_dt == GDN_F32 ? launch_pdl(attn_paged_kernel<float, true>, grid, block, 0, s, a)
                                 : launch_pdl(attn_paged_kernel<bf16, true>, grid, block, 0, s, a);
    return out_dt == GDN_F32 ? launch_pdl(attn_paged_kernel<float, false>, grid, block, 0, s, a)
                             : launch_pdl(attn_paged_kernel<bf16, false>, grid, block, 0, s, a);
}

}  // namespace gdn
