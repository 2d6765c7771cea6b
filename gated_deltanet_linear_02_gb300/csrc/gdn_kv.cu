// gdn_kv.cu -- the input side of the full-attention layers, steps 2-4 of section
// "Full-attention block" of "qwen35moe -- Forward-Pass Design (Pantheon port)"
// and the cache writes that go with them: per-head RMSNorm of q and k, rotation
// of the first 64 of 256 dims, and the rows of the paged cache in bf16 or 4 bits.
//
// One warp per (token, head) row of 256 values, 8 consecutive dims per lane: a
// row is one coalesced 512-byte access, the mean of squares one warp reduction,
// and the rotation's partner dim + 32 is the same register four lanes away. A
// 4-bit group of 64 dims is 8 lanes, whose 8 codes each pack into one 32-bit
// word; a row's 32 words are one 128-byte line of the record.
//
// The kernels are bound by HBM (or, for a few tokens, by launch latency): per
// token and head 512 bytes in, 512 (bf16) or 144 (4 bits) out, and the rotation
// table's 256 bytes per token, shared by its heads through L1.
#include "gdn_async.cuh"
#include "gdn_kv.cuh"

namespace gdn {

constexpr int KV_WARPS = 8;

struct RowSrc {
    const void *p;
    long long row, head;                           // element strides
};

struct InputArgs {
    const float *q_w, *k_w, *rope;
    int n_pos;
    float eps;
    RowSrc q, k, v;
    const int32_t *positions;
    void *q_out, *k_out;                           // dense outputs (k_out: norm entry only)
    void *cache_k, *cache_v;
    int M;
    PagedBatch b;
};

__device__ __forceinline__ void load8(const float *p, float (&x)[8])
{
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const bf16 *p, float (&x)[8])
{
    const uint4 u = *reinterpret_cast<const uint4 *>(p);   // not __ldg: an output may be its own input
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16));
}
__device__ __forceinline__ void load8_in(const float *p, float (&x)[8])
{
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *(reinterpret_cast<const float4 *>(p) + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8_in(const bf16 *p, float (&x)[8]) { load8(p, x); }

__device__ __forceinline__ void store8(float *p, const float (&x)[8])
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(bf16 *p, const float (&x)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// RMSNorm and rotation of a row in fp32. `big` returns the largest magnitude
// that went into any value of this lane's 4-bit group (before or after the
// rotation), which scales the error of the result.
__device__ __forceinline__ void norm_rotate(float (&x)[8], const float *__restrict__ w, const float *__restrict__ rope,
                                            float eps, int lane, float &big, bool &tame)
{
    tame = true;
    if (w != nullptr) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
        ss = warp_sum(ss);
        tame = ss < 1e30f;
        const float r = rsqrtf(fmaf(ss, 1.0f / KV_D, eps));
        float wv[8];
        load8(w + 8 * lane, wv);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * r * wv[i];
    }
    big = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) big = fmaxf(big, fabsf(x[i]));
    if (rope != nullptr) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __shfl_xor_sync(0xffffffffu, x[i], 4);
        if (lane < 8) {                            // dims 0..63: lanes 0-3 the first halves, 4-7 the second
            float c[8], s[8];
            load8(rope + 8 * (lane & 3), c);
            load8(rope + 32 + 8 * (lane & 3), s);
            const float sg = lane < 4 ? -1.0f : 1.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                big = fmaxf(big, fabsf(y[i]));
                x[i] = fmaf(x[i], c[i], sg * y[i] * s[i]);
                big = fmaxf(big, fabsf(x[i]));
            }
        }
    }
}

// The same in 64 bits, from the row as it came.
__device__ __forceinline__ void norm_rotate_f64(const float (&in)[8], double (&x)[8], const float *w, const float *rope,
                                                float eps, int lane)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = in[i];
    if (w != nullptr) {
        double ss = 0.0;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fma(x[i], x[i], ss);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const double r = 1.0 / sqrt(ss * (1.0 / KV_D) + (double)eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * r * (double)__ldg(w + 8 * lane + i);
    }
    if (rope != nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const double y = __shfl_xor_sync(0xffffffffu, x[i], 4);
            if (lane < 8) {
                const double c = __ldg(rope + 8 * (lane & 3) + i), s = __ldg(rope + 32 + 8 * (lane & 3) + i);
                x[i] = lane < 4 ? x[i] * c - y * s : x[i] * c + y * s;
            }
        }
    }
}

// A real number to bf16 in one rounding: to fp32 with the discarded part kept as
// a sticky low bit, then to nearest.
__device__ __forceinline__ float round_bf16(double v)
{
    float f = __double2float_rz(v);
    if ((double)f != v) f = __uint_as_float(__float_as_uint(f) | 1u);
    return to_f(__float2bfloat16_rn(f));
}

struct Quant {
    uint32_t codes;                                // 8 nibbles, dim 0 lowest
    float s, z;
};

// A lane's 8 codes and its group's step and zero, in fp32. `err` bounds the
// distance of every x of the group from the real value it stands for (0: the x
// are exact). Returns whether that error can change nothing: the zero and the
// step round to the same bf16 at both ends of their error intervals, and no
// code's distance from a rounding border is within the error.
__device__ __forceinline__ bool quantise_f32(const float (&x)[8], float err, Quant &q)
{
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    q.z = to_f(__float2bfloat16_rn(lo));
    bool sure = to_f(__float2bfloat16_rn(lo - err)) == to_f(__float2bfloat16_rn(lo + err));
    const float t = (hi - lo) / 15.0f, et = err * (2.0f / 15.0f) + t * 3e-7f;
    q.s = to_f(__float2bfloat16_rn(t));
    sure = sure && to_f(__float2bfloat16_rn(t - et)) == to_f(__float2bfloat16_rn(t + et));
    q.codes = 0;
    if (hi == lo && err == 0.0f) {                 // a constant group: s = 0
        q.s = 0.0f;
        return sure;
    }
    sure = sure && q.s > 1e-30f && q.s < 1e30f;    // away from under- and overflow of 1 / s
    const float inv = 1.0f / q.s;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // d = x - z and the exact rounding error of that subtraction
        const float d = x[i] - q.z, bb = d - x[i];
        const float lost = (x[i] - (d - bb)) + (-q.z - bb);
        const float ed = err + (err > 0.0f || lost != 0.0f ? fabsf(d) * 6e-8f : 0.0f);
        float n = fminf(fmaxf(rintf(d * inv), 0.0f), 15.0f);
        float r = fmaf(-q.s, n, d);                // exact
        // the quotient's own error can leave n one off next to a border
        const float up = r > 0.0f ? 1.0f : -1.0f;
        const float over = fabsf(r) - 0.5f * q.s;
        const bool end = (n == 0.0f && r < 0.0f) || (n == 15.0f && r > 0.0f);
        if (!end) {
            if (over > ed || (over == 0.0f && ed == 0.0f && ((int)n & 1))) n += up;
            else if (!(over < -ed || (over == 0.0f && ed == 0.0f))) sure = false;
        }
        q.codes |= (uint32_t)(int)n << (4 * i);
    }
    return sure;
}

// The definition in 64 bits; a group that holds no finite range reads as NaN.
__device__ __noinline__ void quantise_f64(const double (&x)[8], Quant &q)
{
    double lo = x[0], hi = x[0];
    bool fin = true;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo = fmin(lo, x[i]);
        hi = fmax(hi, x[i]);
        fin = fin && isfinite(x[i]);
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
        lo = fmin(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmax(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        fin = __shfl_xor_sync(0xffffffffu, (int)fin, o) && fin;
    }
    q.codes = 0;
    if (!fin) {
        q.s = 0.0f;
        q.z = __uint_as_float(0x7FC00000u);
        return;
    }
    q.z = round_bf16(lo);
    q.s = round_bf16((hi - lo) / 15.0);
    if (q.s > 0.0f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const double n = fmin(fmax(rint((x[i] - (double)q.z) / (double)q.s), 0.0), 15.0);
            q.codes |= (uint32_t)(int)n << (4 * i);
        }
    }
}

// Warp item: head h of token m; heads 0..15 are queries, 16..17 keys, 18..19
// values. The kernel is instantiated for the heads a call has: NQ queries (0 or
// 16) and NKV (0; 2: keys to k_out; 4: keys and values to the cache).
template <typename TI, typename TO, int NQ, int NKV, bool Q4>
__global__ void __launch_bounds__(KV_WARPS * 32) attn_input_kernel(const InputArgs a)
{
    constexpr int NH = NQ + NKV;
    const int lane = threadIdx.x & 31;
    const long long item = (long long)blockIdx.x * KV_WARPS + (threadIdx.x >> 5);
    const int m = (int)(item / NH), h = (int)(item % NH) + (NQ ? 0 : KV_HQ);
    grid_dep_wait();
    grid_dep_launch();
    if (m >= a.M) return;
    const bool isq = h < KV_HQ, isv = h >= KV_HQ + KV_H;
    const int hh = isq ? h : (isv ? h - KV_HQ - KV_H : h - KV_HQ);

    TokenPlace at = {0, 0};
    if (NKV == 4) {
        at = token_place(a.b, m, lane);
        if (at.seq < 0) return;
    }
    const float *rope = nullptr;
    if (a.rope != nullptr) {
        const int rp = NKV == 4 && a.positions == nullptr ? at.pos : __ldg(a.positions + m);
        if ((unsigned)rp >= (unsigned)a.n_pos) return;
        rope = a.rope + (size_t)rp * GDN_ATTN_ROT_DIM;
    }
    const RowSrc &src = isq ? a.q : (isv ? a.v : a.k);
    float x[8];
    load8_in(static_cast<const TI *>(src.p) + m * src.row + hh * src.head + 8 * lane, x);

    if (isq || NKV == 2) {
        float big;
        bool tame;
        norm_rotate(x, isq ? a.q_w : a.k_w, rope, a.eps, lane, big, tame);
        TO *out = isq ? static_cast<TO *>(a.q_out) + ((size_t)m * KV_HQ + hh) * KV_D
                      : static_cast<TO *>(a.k_out) + ((size_t)m * KV_H + hh) * KV_D;
        store8(out + 8 * lane, x);
        return;
    }
    const int page = cache_page(a.b, at.seq, at.pos);
    if (page < 0) return;
    const int off = at.pos & (a.b.page - 1);
    if (!Q4) {
        float big;
        bool tame;
        if (!isv) norm_rotate(x, a.k_w, rope, a.eps, lane, big, tame);
        bf16 *dst = static_cast<bf16 *>(isv ? a.cache_v : a.cache_k) + row_bf16(a.b, page, hh, off);
        store8(dst + 8 * lane, x);
        return;
    }
    float in[8], err = 0.0f;
    bool sure = true;
#pragma unroll
    for (int i = 0; i < 8; ++i) in[i] = x[i];
    if (!isv && (a.k_w != nullptr || rope != nullptr)) {
        // Error of a normed and rotated value: the mean of squares (8 + 5
        // additions, halved by the root), rsqrt (2 ulp), two products, and the
        // rotation's two products and one sum, each relative to `big`: below
        // 7e-7 big in all. 2e-6 big leaves a factor of two and a half.
        float big;
        norm_rotate(x, a.k_w, rope, a.eps, lane, big, sure);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
        err = 2e-6f * big;
    }
    float far = 0.0f;                              // infinities and NaN are the 64-bit form's
#pragma unroll
    for (int i = 0; i < 8; ++i) far += fabsf(x[i]);
    Quant q;
    sure = quantise_f32(x, err, q) && sure && far < 1e30f;
    if (!__all_sync(0xffffffffu, sure)) {
        double xd[8];
        norm_rotate_f64(in, xd, isv ? nullptr : a.k_w, isv ? nullptr : rope, a.eps, lane);
        quantise_f64(xd, q);
    }
    unsigned char *rec = static_cast<unsigned char *>(a.cache_k) + record_of(a.b, page, hh, off);
    const int r = off & (REC_ROWS - 1), g = lane >> 3, c = lane & 7;
    *reinterpret_cast<uint32_t *>(rec + (isv ? REC_V : 0u) + r * 128 + c * 16 + g * 4) = q.codes;
    if (c == 0)
        *reinterpret_cast<uint32_t *>(rec + (isv ? REC_VSZ : REC_KSZ) + r * 16 + g * 4) =
            (__float_as_uint(q.s) >> 16) | (__float_as_uint(q.z) & 0xFFFF0000u);
}

template <typename TI, typename TO, int NQ, int NKV, bool Q4>
static cudaError_t launch_input(const InputArgs &a, cudaStream_t s)
{
    const long long items = (long long)a.M * (NQ + NKV);
    return launch_pdl(attn_input_kernel<TI, TO, NQ, NKV, Q4>, dim3((unsigned)((items + KV_WARPS - 1) / KV_WARPS)),
                      dim3(KV_WARPS * 32), 0, s, a);
}

cudaError_t launch_qk_norm_rope(const gdn_attn_params *p, const void *q, long long q_row, long long q_head,
                                const void *k, long long k_row, long long k_head, const int32_t *positions, int M,
                                void *q_out, void *k_out, gdn_dtype act, gdn_dtype out_dt, cudaStream_t s)
{
    InputArgs a = {p->q_norm_w, p->k_norm_w, p->rope, p->n_pos, p->norm_eps, {q, q_row, q_head}, {k, k_row, k_head},
                   {}, positions, q_out, k_out, nullptr, nullptr, M, {}};
    const bool fi = act == GDN_F32, fo = out_dt == GDN_F32;
    if (k == nullptr) {
        if (fi) return fo ? launch_input<float, float, KV_HQ, 0, false>(a, s) : launch_input<float, bf16, KV_HQ, 0, false>(a, s);
        return fo ? launch_input<bf16, float, KV_HQ, 0, false>(a, s) : launch_input<bf16, bf16, KV_HQ, 0, false>(a, s);
    }
    if (fi) return fo ? launch_input<float, float, KV_HQ, KV_H, false>(a, s) : launch_input<float, bf16, KV_HQ, KV_H, false>(a, s);
    return fo ? launch_input<bf16, float, KV_HQ, KV_H, false>(a, s) : launch_input<bf16, bf16, KV_HQ, KV_H, false>(a, s);
}

cudaError_t launch_kv_append(const gdn_attn_params *p, const gdn_paged_batch *b, const gdn_kv_cache *c, const void *k,
                             long long k_row, long long k_head, const void *v, long long v_row, long long v_head,
                             const void *q, long long q_row, long long q_head, void *q_out, const int32_t *positions,
                             gdn_dtype act, cudaStream_t s)
{
    InputArgs a = {p->q_norm_w, p->k_norm_w, p->rope, p->n_pos, p->norm_eps, {q, q_row, q_head}, {k, k_row, k_head},
                   {v, v_row, v_head}, positions, q_out, nullptr, c->k, c->v, b->M, paged_batch(*b, *c)};
    const bool f = act == GDN_F32, four = c->format == GDN_KV_Q4;
    if (q == nullptr) {
        if (f) return four ? launch_input<float, bf16, 0, 2 * KV_H, true>(a, s) : launch_input<float, bf16, 0, 2 * KV_H, false>(a, s);
        return four ? launch_input<bf16, bf16, 0, 2 * KV_H, true>(a, s) : launch_input<bf16, bf16, 0, 2 * KV_H, false>(a, s);
    }
    if (f) return four ? launch_input<float, bf16, KV_HQ, 2 * KV_H, true>(a, s) : launch_input<float, bf16, KV_HQ, 2 * KV_H, false>(a, s);
    return four ? launch_input<bf16, bf16, KV_HQ, 2 * KV_H, true>(a, s) : launch_input<bf16, bf16, KV_HQ, 2 * KV_H, false>(a, s);
}

// Reads rows back: the same warp layout, values z + s c in fp32 (s c is exact:
// 8 x 4 bits), one rounding to the output type.
template <typename TO, bool Q4>
__global__ void __launch_bounds__(KV_WARPS * 32) kv_gather_kernel(const PagedBatch b, const void *ck, const void *cv,
                                                                  TO *k_out, TO *v_out)
{
    const int lane = threadIdx.x & 31;
    const long long item = (long long)blockIdx.x * KV_WARPS + (threadIdx.x >> 5);
    const int m = (int)(item >> 2), h = (int)item & 1;
    const bool isv = (item & 2) != 0;
    grid_dep_wait();
    grid_dep_launch();
    TO *out = isv ? v_out : k_out;
    if (m >= b.M || out == nullptr) return;
    const TokenPlace at = token_place(b, m, lane);
    if (at.seq < 0) return;
    const int page = cache_page(b, at.seq, at.pos), off = at.pos & (b.page - 1);
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (page >= 0) {
        if (!Q4) {
            load8(static_cast<const bf16 *>(isv ? cv : ck) + row_bf16(b, page, h, off) + 8 * lane, x);
        } else {
            const unsigned char *rec = static_cast<const unsigned char *>(ck) + record_of(b, page, h, off);
            const int r = off & (REC_ROWS - 1), g = lane >> 3, c = lane & 7;
            const uint32_t w = *reinterpret_cast<const uint32_t *>(rec + (isv ? REC_V : 0u) + r * 128 + c * 16 + g * 4);
            const uint32_t sz = *reinterpret_cast<const uint32_t *>(rec + (isv ? REC_VSZ : REC_KSZ) + r * 16 + g * 4);
            const float s = __uint_as_float(sz << 16), z = __uint_as_float(sz & 0xFFFF0000u);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = fmaf(s, (float)((w >> (4 * i)) & 15u), z);
        }
    }
    store8(out + ((size_t)m * KV_H + h) * KV_D + 8 * lane, x);
}

cudaError_t launch_kv_gather(const gdn_paged_batch *b, const gdn_kv_cache *c, void *k_out, void *v_out,
                             gdn_dtype out_dt, cudaStream_t s)
{
    const PagedBatch pb = paged_batch(*b, *c);
    const dim3 grid((unsigned)(((long long)b->M * 2 * KV_H + KV_WARPS - 1) / KV_WARPS)), block(KV_WARPS * 32);
    const void *ck = c->k, *cv = c->v;
    if (c->format == GDN_KV_Q4)
        return out_dt == GDN_F32 ? launch_pdl(kv_gather_kernel<float, true>, grid, block, 0, s, pb, ck, cv, (float *)k_out, (float *)v_out)
                                 : launch_pdl(kv_gather_kernel<bf16, true>, grid, block, 0, s, pb, ck, cv, (bf16 *)k_out, (bf16 *)v_out);
    return out_dt == GDN_F32 ? launch_pdl(kv_gather_kernel<float, false>, grid, block, 0, s, pb, ck, cv, (float *)k_out, (float *)v_out)
                             : launch_pdl(kv_gather_kernel<bf16, false>, grid, block, 0, s, pb, ck, cv, (bf16 *)k_out, (bf16 *)v_out);
}

}  // namespace gdn
