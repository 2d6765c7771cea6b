// gdn_kv.cu -- the input side of the full-attention layers, steps 2-4 of section
// "Full-attention block" of "qwen35moe -- Forward-Pass Design (Pantheon port)"
// and the cache writes that go with them: per-head RMSNorm of q and k, rotation
// of the first 64 of 256 dims, and the rows of the paged cache in bf16 or 4 bits.
//
// A (token, head) row of 256 values is one warp's, 8 consecutive dims per lane: a
// row is one coalesced 512-byte access, the mean of squares one warp reduction, and
// the rotation's partner dim + 32 is the same register four lanes away. A 4-bit
// group of 64 dims is 8 lanes, whose 8 codes each pack into one 32-bit word; a
// row's 32 words are one 128-byte line of the record.
//
// Per token and head 512 bytes go in, 512 (bf16) or 144 (4 bits) out, and the rotation
// table's 256 bytes per token. With many tokens a warp takes four rows of one token, whose
// loads all start before the token's place in the cache is looked up (a chain of
// dependent reads); with few, one row, so that more SMs share them. Few tokens are bound
// by latency, many by bytes and instructions together (two thirds of the issue slots
// while an SM is active). Measured, buffers in turn beyond L2: norms and rotation of
// 4,096 tokens 16.9 us (4.5 TB/s; a copy of as many bytes at full rate takes 11.3; 15.8
// in L2), bf16 append with queries 17.8 us (4.7 TB/s), 4-bit append 14.4 us: there the
// exact codes are bound by instructions, 489 per row and warp.
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

__device__ __forceinline__ float sum_squares(const float (&x)[8])
{
    const float s0 = fmaf(x[1], x[1], x[0] * x[0]), s1 = fmaf(x[3], x[3], x[2] * x[2]);
    const float s2 = fmaf(x[5], x[5], x[4] * x[4]), s3 = fmaf(x[7], x[7], x[6] * x[6]);
    return warp_sum((s0 + s1) + (s2 + s3));
}
// The mean of a row's squares plus eps. Where the squares leave fp32's normal numbers
// (rows near 1e-15 and eps below 1e-30, or near 1e14) the row is scaled by 2^100 or
// 2^-100 and the mean is that of the scaled row, by which the norm stays the same.
// `far` says that this is so; all lanes agree, as warp_sum gives them the same bits.
__device__ __forceinline__ float mean_square(const float (&x)[8], float eps, bool &far)
{
    const float ss = sum_squares(x), v = fmaf(ss, 1.0f / KV_D, eps);
    far = !(ss < 1e30f && v > 1e-30f);
    return v;
}
__device__ __forceinline__ float mean_square_far(float (&x)[8], float eps)
{
    const float f = sum_squares(x) < 1e30f ? 0x1p100f : 0x1p-100f;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= f;
    return fmaf(sum_squares(x), 1.0f / KV_D, eps * f * f);
}

// RMSNorm and rotation of a row in fp32. `tol` returns a bound of each value's error,
// in units of 2^-24 of what went into it: the mean of squares 10 (a rounded square, a
// tree of 8 additions, and eps), halved by the root, the refined root 1.5, two products
// 2: 8.5 of |x|; a rotated one three roundings more, 11.5 of |x c| + |y s|. In bf16 rows
// (TI) the squares are exact, which is 0.5 less. `tame`: the mean of squares is such that
// this holds.
template <typename TI>
__device__ __forceinline__ void norm_rotate(float (&x)[8], const float *__restrict__ w, const float *__restrict__ rope,
                                            float eps, int lane, float (&tol)[8], bool &tame)
{
    tame = true;
    if (w != nullptr) {
        bool far;
        float v = mean_square(x, eps, far);
        if (far) v = mean_square_far(x, eps);
        const float r0 = rsqrtf(v);
        const float r = fmaf(r0 * 0.5f, fmaf(-v * r0, r0, 1.0f), r0);   // one Newton step: the last bit
        tame = !far;
        float wv[8];
        load8(w + 8 * lane, wv);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * r * wv[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) tol[i] = (sizeof(TI) == 2 ? 4.8e-7f : 5.1e-7f) * fabsf(x[i]);
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
                const float t = sg * y[i] * s[i];
                tol[i] = (sizeof(TI) == 2 ? 6.6e-7f : 6.9e-7f) * (fabsf(x[i] * c[i]) + fabsf(t));
                x[i] = fmaf(x[i], c[i], t);
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

// ---- pairs of fp32 numbers (h + l, |l| at most half a last place of h): 48 bits
// by Dekker's and Knuth's exact sums and products, several times as fast as 64-bit
// arithmetic here (2 fused multiply-adds per cycle and SM). For magnitudes whose
// low parts stay normal; others take the 64-bit form below.
struct Pair {
    float h, l;
};
__device__ __forceinline__ Pair two_sum(float a, float b)
{
    const float s = a + b, bb = s - a;
    return Pair{s, (a - (s - bb)) + (b - bb)};
}
__device__ __forceinline__ Pair quick_sum(float a, float b)   // |a| >= |b|
{
    const float s = a + b;
    return Pair{s, b - (s - a)};
}
__device__ __forceinline__ Pair add(Pair x, Pair y)
{
    const Pair s = two_sum(x.h, y.h), t = two_sum(x.l, y.l), u = quick_sum(s.h, s.l + t.h);
    return quick_sum(u.h, u.l + t.l);
}
__device__ __forceinline__ Pair mul(Pair x, float f)
{
    const float p = x.h * f;
    return quick_sum(p, fmaf(x.l, f, fmaf(x.h, f, -p)));
}
__device__ __forceinline__ Pair mul(Pair x, Pair y)
{
    const float p = x.h * y.h;
    return quick_sum(p, fmaf(x.l, y.h, fmaf(x.h, y.l, fmaf(x.h, y.h, -p))));
}
__device__ __forceinline__ Pair shfl_xor(Pair x, int o)
{
    return Pair{__shfl_xor_sync(0xffffffffu, x.h, o), __shfl_xor_sync(0xffffffffu, x.l, o)};
}
__device__ __forceinline__ bool below(Pair x, Pair y) { return x.h < y.h || (x.h == y.h && x.l < y.l); }
// To bf16 in one rounding: toward zero to fp32 with the rest as a sticky low bit, then to nearest.
__device__ __forceinline__ float round_bf16(Pair x)
{
    uint32_t u = __float_as_uint(x.h);
    if (x.l != 0.0f) u = (u - ((x.l > 0.0f) != (x.h > 0.0f) ? 1u : 0u)) | 1u;
    return to_f(__float2bfloat16_rn(__uint_as_float(u)));
}

// RMSNorm and rotation of a row in pairs, from the row as it came.
__device__ __forceinline__ void norm_rotate_pair(const float (&in)[8], Pair (&x)[8], const float *w, const float *rope,
                                                 float eps, int lane)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = Pair{in[i], 0.0f};
    if (w != nullptr) {
        Pair sq[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) sq[i] = mul(x[i], in[i]);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < o; ++i) sq[i] = add(sq[i], sq[i + o]);
        Pair ss = sq[0];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss = add(ss, shfl_xor(ss, o));
        const Pair v = add(mul(ss, 1.0f / KV_D), Pair{eps, 0.0f});
        // v^-1/2: one step of r (1 + e / 2 + 3 e^2 / 8) with e = 1 - v r^2 from the hardware's r
        const float r0 = rsqrtf(v.h);
        const Pair t = mul(mul(v, r0), r0);
        const float e = (1.0f - t.h) - t.l;
        const Pair r = quick_sum(r0, r0 * fmaf(0.375f * e, e, 0.5f * e));
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = mul(mul(r, __ldg(w + 8 * lane + i)), in[i]);
    }
    if (rope != nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const Pair y = shfl_xor(x[i], 4);
            if (lane < 8) {
                const float c = __ldg(rope + 8 * (lane & 3) + i), s = __ldg(rope + 32 + 8 * (lane & 3) + i);
                x[i] = add(mul(x[i], c), mul(y, lane < 4 ? -s : s));
            }
        }
    }
}

// A real number to bf16 in one rounding, as above.
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

// A lane's 8 codes and its group's step and zero, in fp32. `tol` bounds the distance
// of each x from the real value it stands for, `err` those of the whole group. Returns
// whether neither that nor the arithmetic's own error can change anything: the zero
// and the step round to the same bf16 at both ends of their error intervals (`range`),
// and every x lies inside its code's interval by more than its error and the rounding
// of x - z. (That the product with 1 / s rounds to a neighbour's code shows as x
// outside the interval.) Rounding to an integer is adding 1.5 2^23; four codes are
// joined in fp32, whose 24 bits hold them exactly.
__device__ __forceinline__ bool quantise_f32(const float (&x)[8], const float (&tol)[8], float err, Quant &q, bool &range)
{
    float lo = fminf(fminf(fminf(x[0], x[1]), fminf(x[2], x[3])), fminf(fminf(x[4], x[5]), fminf(x[6], x[7])));
    float hi = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    q.z = to_f(__float2bfloat16_rn(lo));
    const float t = (hi - lo) * (1.0f / 15.0f), et = err * (2.0f / 15.0f) + t * 3e-7f;
    q.s = to_f(__float2bfloat16_rn(t));
    q.codes = 0;
    if (hi == lo && err == 0.0f && (lo == 0.0f || fabsf(lo) > 1e-30f)) {   // a constant group: s = 0 (not where `tol` underflows)
        q.s = 0.0f;
        return range = true;
    }
    const float inv = __fdividef(1.0f, q.s), half = 0.5f * q.s, magic = 12582912.0f;
    float inside = q.s, n[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float d = x[i] - q.z;
        n[i] = fmaf(d, inv, magic) - magic;
        inside = fminf(inside, half - fabsf(fmaf(-q.s, n[i], d)) - fmaf(1.2e-7f, fabsf(d), tol[i]));
        n[i] = fminf(fmaxf(n[i], 0.0f), 15.0f);
    }
    const float a = fmaf(4096.0f, n[3], fmaf(256.0f, n[2], fmaf(16.0f, n[1], n[0])));
    const float b = fmaf(4096.0f, n[7], fmaf(256.0f, n[6], fmaf(16.0f, n[5], n[4])));
    q.codes = __byte_perm(__float_as_uint(a + 8388608.0f), __float_as_uint(b + 8388608.0f), 0x5410);   // low 16 bits of each
    range = to_f(__float2bfloat16_rn(lo - err)) == to_f(__float2bfloat16_rn(lo + err)) &&
            to_f(__float2bfloat16_rn(t - et)) == to_f(__float2bfloat16_rn(t + et)) && q.s > 1e-30f && q.s < 1e30f;
    return range && inside > 0.0f;
}

// Exact x (err = 0) next to a border: the same with every comparison exact in fp32,
// ties to the even code. Returns whether that was possible.
__device__ __forceinline__ bool quantise_exact(const float (&x)[8], Quant &q)
{
    const float inv = 1.0f / q.s, half = 0.5f * q.s;
    bool sure = true;
    q.codes = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // d = x - z and the exact rounding error of that subtraction, which has to be nothing
        const float d = x[i] - q.z, bb = d - x[i];
        const bool exact = (x[i] - (d - bb)) + (-q.z - bb) == 0.0f;
        float n = fminf(fmaxf(rintf(d * inv), 0.0f), 15.0f);
        const float r = fmaf(-q.s, n, d), over = fabsf(r) - half;   // both exact
        const bool end = (n == 0.0f && r < 0.0f) || (n == 15.0f && r > 0.0f);
        if (!end && (over > 0.0f || (over == 0.0f && ((int)n & 1)))) n += r > 0.0f ? 1.0f : -1.0f;
        sure = sure && (exact || fabsf(over) > 1e-6f * fabsf(d));
        q.codes |= (uint32_t)(int)n << (4 * i);
    }
    return sure;
}

// The definition in pairs.
__device__ __noinline__ void quantise_pair(const Pair (&x)[8], Quant &q)
{
    Pair lo = x[0], hi = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        if (below(x[i], lo)) lo = x[i];
        if (below(hi, x[i])) hi = x[i];
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
        const Pair a = shfl_xor(lo, o), b = shfl_xor(hi, o);
        if (below(a, lo)) lo = a;
        if (below(hi, b)) hi = b;
    }
    q.z = round_bf16(lo);
    const Pair d = add(hi, Pair{-lo.h, -lo.l});
    const float t = d.h / 15.0f;
    q.s = round_bf16(quick_sum(t, (fmaf(-15.0f, t, d.h) + d.l) / 15.0f));
    q.codes = 0;
    if (q.s == 0.0f) return;
    const float inv = 1.0f / q.s, half = 0.5f * q.s;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const Pair a = add(x[i], Pair{-q.z, 0.0f});
        float n = fminf(fmaxf(rintf(a.h * inv), 0.0f), 15.0f);
        const Pair r = two_sum(fmaf(-q.s, n, a.h), a.l);
        const float up = r.h > 0.0f ? 1.0f : -1.0f, over = (fabsf(r.h) - half) + up * r.l;
        const bool end = (n == 0.0f && r.h < 0.0f) || (n == 15.0f && r.h > 0.0f);
        if (!end && (over > 0.0f || (over == 0.0f && ((int)n & 1)))) n += up;
        q.codes |= (uint32_t)(int)n << (4 * i);
    }
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

// One K or V row in registers to its 4-bit place: fp32 where its error can change
// nothing, else in pairs, or in 64 bits where pairs leave their range.
template <typename TI>
__device__ __forceinline__ void store_row_q4(const InputArgs &a, const float (&in)[8], bool isv, const float *rope, int page,
                                             int head, int off, int lane)
{
    float x[8], tol[8] = {}, err = 0.0f;
    bool tame = true;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = in[i];
    if (!isv && (a.k_w != nullptr || rope != nullptr)) {
        norm_rotate<TI>(x, a.k_w, rope, a.eps, lane, tol, tame);
#pragma unroll
        for (int i = 0; i < 8; ++i) err = fmaxf(err, tol[i]);
        tame = tame && ((tol[0] + tol[1]) + (tol[2] + tol[3])) + ((tol[4] + tol[5]) + (tol[6] + tol[7])) < 1e30f;   // no NaN
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) err = fmaxf(err, __shfl_xor_sync(0xffffffffu, err, o));
    }
    float all = 0.0f;                              // of the row as it came; infinities and NaN are the 64-bit form's
#pragma unroll
    for (int i = 0; i < 8; ++i) all += fabsf(in[i]);
    Quant q;
    bool range, sure = quantise_f32(x, tol, err, q, range) && tame && all < 1e30f;
    // `err` is a group's own, so groups of one row may differ in it: the votes are taken by the whole warp, and
    // only what has no exchange between lanes depends on it.
    if (!__all_sync(0xffffffffu, sure)) {
        // Exact values that are next to a border are mostly ties, which fp32 can settle.
        if (!sure && err == 0.0f && tame && range && all < 1e30f) sure = quantise_exact(x, q);
        const bool mid = tame && all < 1e12f && (all > 1e-10f || all == 0.0f) && err < 5e5f && (err > 5e-17f || err == 0.0f) &&
                         q.s < 1e12f && (q.s > 1e-12f || q.s == 0.0f);
        if (__all_sync(0xffffffffu, sure)) {
        } else if (__all_sync(0xffffffffu, mid)) {
            Pair xp[8];
            norm_rotate_pair(in, xp, isv ? nullptr : a.k_w, isv ? nullptr : rope, a.eps, lane);
            quantise_pair(xp, q);
        } else {
            double xd[8];
            norm_rotate_f64(in, xd, isv ? nullptr : a.k_w, isv ? nullptr : rope, a.eps, lane);
            quantise_f64(xd, q);
        }
    }
    unsigned char *rec = static_cast<unsigned char *>(a.cache_k) + record_of(a.b, page, head, off);
    const int r = off & (REC_ROWS - 1), g = lane >> 3, c = lane & 7;
    *reinterpret_cast<uint32_t *>(rec + (isv ? REC_V : 0u) + r * 128 + c * 16 + g * 4) = q.codes;
    if (c == 0)
        *reinterpret_cast<uint32_t *>(rec + (isv ? REC_VSZ : REC_KSZ) + r * 16 + g * 4) =
            (__float_as_uint(q.s) >> 16) | (__float_as_uint(q.z) & 0xFFFF0000u);
}

// Few rows: one warp per row. Heads 0..15 of a token are queries (NQ 0 or 16), then
// NKV rows: 2, its keys for k_out, or 4, its keys and values for the cache.
template <typename TI, typename TO, int NQ, int NKV, bool Q4>
__global__ void __launch_bounds__(KV_WARPS * 32) attn_input_few_kernel(const InputArgs a)
{
    constexpr int NH = NQ + NKV;
    const int lane = threadIdx.x & 31;
    const int item = blockIdx.x * KV_WARPS + (threadIdx.x >> 5);   // below 2^31: the host sends more rows to the other kernel
    const int m = item / NH, u = item % NH;
    grid_dep_wait();
    grid_dep_launch();
    if (m >= a.M) return;
    const bool isq = u < NQ, isv = u >= NQ + KV_H;
    const int h = isq ? u : (isv ? u - NQ - KV_H : u - NQ);
    const RowSrc src = isq ? a.q : (isv ? a.v : a.k);
    float x[8];
    load8_in(static_cast<const TI *>(src.p) + m * src.row + h * src.head + 8 * lane, x);
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
    if (NKV == 4 && !isq) {
        const int page = cache_page(a.b, at.seq, at.pos), off = at.pos & (a.b.page - 1);
        if (page < 0) return;
        if (Q4) {
            store_row_q4<TI>(a, x, isv, rope, page, h, off, lane);
            return;
        }
        float tol[8];
        bool tame;
        if (!isv) norm_rotate<TI>(x, a.k_w, rope, a.eps, lane, tol, tame);
        store8(static_cast<bf16 *>(isv ? a.cache_v : a.cache_k) + row_bf16(a.b, page, h, off) + 8 * lane, x);
        return;
    }
    float tol[8];
    bool tame;
    norm_rotate<TI>(x, isq ? a.q_w : a.k_w, rope, a.eps, lane, tol, tame);
    store8(isq ? static_cast<TO *>(a.q_out) + ((size_t)m * KV_HQ + h) * KV_D + 8 * lane
               : static_cast<TO *>(a.k_out) + ((size_t)m * KV_H + h) * KV_D + 8 * lane, x);
}

// Many rows: a fixed grid whose warps each walk a stretch of tokens with one unit
// of heads (QR queries, or the token's keys and values; one of those in 4 bits).
// A warp looks up the places of 32 tokens at a time, one per lane, and starts the
// next token's rows and rotation before it works on the current one's.
template <typename TI> struct Raw8;
template <> struct Raw8<bf16> {
    uint4 v;
    __device__ __forceinline__ void load(const bf16 *p) { v = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void get(float (&x)[8]) const
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16));
    }
};
template <> struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = reinterpret_cast<const float4 *>(p)[0];
        b = reinterpret_cast<const float4 *>(p)[1];
    }
    __device__ __forceinline__ void get(float (&x)[8]) const
    {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
};

// The row times r and the weights, and the rotation (lanes 0-7's), from registers.
__device__ __forceinline__ void norm_rotate_regs(float (&x)[8], bool norm, float r, const float (&w)[8], bool rot,
                                                 const float (&c)[8], const float (&s)[8], int lane)
{
    if (norm)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
    if (rot) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float y = __shfl_xor_sync(0xffffffffu, x[i], 4);
            x[i] = lane < 8 ? fmaf(x[i], c[i], (lane < 4 ? -y : y) * s[i]) : x[i];
        }
    }
}

constexpr int QR = 4;                             // queries per warp and token

// One unit over the tokens [m0, m1): N rows of each, `first` the first of them
// (queries 0..15; k0, k1, v0, v1).
template <typename TI, typename TO, int NKV, bool Q4, bool ISQ, int N>
__device__ __forceinline__ void walk_tokens(const InputArgs &a, int first, int m0, int m1, int lane)
{
    const bool rot = a.rope != nullptr;
    const float *wp = ISQ ? a.q_w : a.k_w;
    float w[8] = {}, c[8] = {}, s[8] = {};
    if (wp != nullptr) load8(wp + 8 * lane, w);
    Raw8<TI> cur[N], nxt[N];
    auto load = [&](Raw8<TI> (&raw)[N], int m) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int r = first + i;
            const RowSrc src = ISQ ? a.q : (r < KV_H ? a.k : a.v);
            raw[i].load(static_cast<const TI *>(src.p) + m * src.row + (ISQ || r < KV_H ? r : r - KV_H) * src.head + 8 * lane);
        }
    };
    load(nxt, m0);
    for (int base = m0; base < m1; base += 32) {
        // places of 32 tokens, one per lane: rotation row (-1: the token is padding), page (-1: none), row in the page
        const int mine = min(base + lane, m1 - 1);
        int seq = 0, pos = 0, page = 0, rp = 0;
        if (NKV == 4) {
            seq = mine < a.b.B || a.b.cu != nullptr ? mine : -1;
            if (a.b.cu != nullptr) {               // the number of entries cu[1..B] at or below the row
                int lo = 0, hi = a.b.B;
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (__ldg(a.b.cu + mid) <= mine) lo = mid;
                    else hi = mid - 1;
                }
                seq = lo < a.b.B ? lo : -1;
            }
            if (seq >= 0) {
                pos = __ldg(a.b.ctx + seq) - (a.b.cu != nullptr ? __ldg(a.b.cu + seq + 1) - mine : 1);
                page = ISQ ? 0 : cache_page(a.b, seq, pos);
            }
        }
        if (a.rope != nullptr) rp = NKV == 4 && a.positions == nullptr ? pos : __ldg(a.positions + mine);
        if (seq < 0 || (a.rope != nullptr && (unsigned)rp >= (unsigned)a.n_pos)) rp = -1;
        const int n = min(32, m1 - base);
        float cn[8] = {}, sn[8] = {};
        auto turn = [&](int k) {                   // the rotation of token base + k
            const int r = __shfl_sync(0xffffffffu, rp, k);
            if (rot && r >= 0 && lane < 8) {
                const float *row = a.rope + (size_t)r * GDN_ATTN_ROT_DIM + 8 * (lane & 3);
                load8(row, cn);
                load8(row + 32, sn);
            }
        };
        auto store = [&](int i, int m, int pg, int off, const float (&x)[8]) {
            const int row = first + i, h = ISQ || row < KV_H ? row : row - KV_H;
            if (ISQ) store8(static_cast<TO *>(a.q_out) + ((size_t)m * KV_HQ + h) * KV_D + 8 * lane, x);
            else if (NKV == 2) store8(static_cast<TO *>(a.k_out) + ((size_t)m * KV_H + h) * KV_D + 8 * lane, x);
            else store8(static_cast<bf16 *>(row >= KV_H ? a.cache_v : a.cache_k) + row_bf16(a.b, pg, h, off) + 8 * lane, x);
        };
        uint32_t left = 0u;                        // tokens left for the end
        turn(0);
        for (int k = 0; k < n; ++k) {
            const int m = base + k;
#pragma unroll
            for (int i = 0; i < N; ++i) cur[i] = nxt[i];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                c[i] = cn[i];
                s[i] = sn[i];
            }
            if (m + 1 < m1) load(nxt, m + 1);
            if (k + 1 < n) turn(k + 1);
            const int r = __shfl_sync(0xffffffffu, rp, k), pg = __shfl_sync(0xffffffffu, page, k);
            const int off = __shfl_sync(0xffffffffu, pos, k) & (a.b.page - 1);
            if (r < 0 || pg < 0) continue;
            // The norms of all rows first, then one test whether squares of any leave fp32 (see mean_square): such a
            // token is left as it is until the end, as a branch per row would keep the rows from running side by
            // side (norms of 4,096 tokens 18.4 instead of 16.9 us).
            float root[N] = {};
            if (!(Q4 && !ISQ) && wp != nullptr) {
                bool any = false;
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (ISQ || first + i < KV_H) {
                        float x[8];
                        bool far;
                        cur[i].get(x);
                        root[i] = rsqrtf(mean_square(x, a.eps, far));
                        any = any || far;
                    }
                if (any) {
                    left |= 1u << k;
                    continue;
                }
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float x[8];
                cur[i].get(x);
                if (Q4 && !ISQ) {
                    const int row = first + i;
                    store_row_q4<TI>(a, x, row >= KV_H, a.rope != nullptr ? a.rope + (size_t)r * GDN_ATTN_ROT_DIM : nullptr, pg,
                                 row < KV_H ? row : row - KV_H, off, lane);
                    continue;
                }
                if (ISQ || first + i < KV_H) norm_rotate_regs(x, wp != nullptr, root[i], w, rot, c, s, lane);
                store(i, m, pg, off, x);
            }
        }
        if (Q4 && !ISQ) continue;
        for (; left != 0u; left &= left - 1) {
            const uint32_t k = __ffs(left) - 1;
            turn(k);
            load(cur, base + k);
            const int pg = __shfl_sync(0xffffffffu, page, k), off = __shfl_sync(0xffffffffu, pos, k) & (a.b.page - 1);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float x[8];
                bool far;
                cur[i].get(x);
                if (ISQ || first + i < KV_H) {
                    float v = mean_square(x, a.eps, far);
                    if (far) v = mean_square_far(x, a.eps);
                    norm_rotate_regs(x, true, rsqrtf(v), w, rot, cn, sn, lane);
                }
                store(i, base + k, pg, off, x);
            }
        }
    }
}

// CTAs per SM: two hold four queries a warp and the next token's; keys and values
// alone into 4 bits are bound by instructions, and hide them better with more warps.
constexpr int input_ctas(int nq, bool q4) { return nq == 0 && q4 ? 3 : 2; }

template <typename TI, typename TO, int NQ, int NKV, bool Q4>
__global__ void __launch_bounds__(KV_WARPS * 32, input_ctas(NQ, Q4)) attn_input_kernel(const InputArgs a)
{
    constexpr int UQ = NQ / QR, UK = Q4 ? NKV : NKV > 0 ? 1 : 0, U = UQ + UK;
    const int lane = threadIdx.x & 31, gw = blockIdx.x * KV_WARPS + (threadIdx.x >> 5);
    const int stretches = (int)gridDim.x * KV_WARPS / U, at = gw / U, u = gw % U;
    grid_dep_wait();
    grid_dep_launch();
    const int per = (a.M + stretches - 1) / stretches;
    const int m0 = min((long long)at * per, (long long)a.M), m1 = min(m0 + per, a.M);
    if (at >= stretches || m0 >= m1) return;
    if (u < UQ) walk_tokens<TI, TO, NKV, Q4, true, QR>(a, u * QR, m0, m1, lane);
    else if (Q4) walk_tokens<TI, TO, NKV, Q4, false, 1>(a, u - UQ, m0, m1, lane);
    else if (NKV > 0) walk_tokens<TI, TO, NKV, Q4, false, NKV == 4 ? 4 : 2>(a, 0, m0, m1, lane);
}

// Rows up to which one warp takes one row, two waves of 48 warps on each of 152 SMs,
// and above which warps walk. Both sides, us, in L2: norms of 512 tokens (9,216 rows) 4.1
// against 4.9, 811 (14,598 rows) 5.1 both, 4,096 18.0 against 15.8; bf16 append with
// queries 512 5.4 both, 811 6.8 against 5.5, 4,096 24.6 against 16.9; 4-bit append 1,024
// (4,096 rows) 6.9 against 8.6, 2,048 9.7 against 10.3, 4,096 14.6 against 14.0. Keys and
// values into bf16 pages are copies but for the norm, and gain from the walk's loads
// ahead sooner: 512 tokens 3.3 both, 2,048 5.5 against 3.9.
constexpr long long few_rows(int nq, int nkv, bool q4) { return nq == 0 && nkv == 4 && !q4 ? 2048 : 2 * 152 * 48; }

template <typename TI, typename TO, int NQ, int NKV, bool Q4>
static cudaError_t launch_input(const InputArgs &a, cudaStream_t s)
{
    const long long rows = (long long)a.M * (NQ + NKV);
    if (rows <= few_rows(NQ, NKV, Q4))
        return launch_pdl(attn_input_few_kernel<TI, TO, NQ, NKV, Q4>, dim3((unsigned)((rows + KV_WARPS - 1) / KV_WARPS)),
                          dim3(KV_WARPS * 32), 0, s, a);
    return launch_pdl(attn_input_kernel<TI, TO, NQ, NKV, Q4>, dim3(input_ctas(NQ, Q4) * 152), dim3(KV_WARPS * 32),
                      0, s, a);
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
// 8 x 4 bits), one rounding to the output type. A warp takes a token's k0, k1, v0, v1:
// 4,096 tokens in bf16 out of 4-bit pages 4.2 us, 3.5 in L2 (one row per warp a third
// more), out of bf16 pages 4.2; 2^20 tokens 414 us (6.6 TB/s) and 617 us (7.0 TB/s).
template <typename TO, bool Q4>
__global__ void __launch_bounds__(KV_WARPS * 32) kv_gather_kernel(const PagedBatch b, const void *ck, const void *cv,
                                                                  TO *k_out, TO *v_out)
{
    const int lane = threadIdx.x & 31;
    const int m = blockIdx.x * KV_WARPS + (threadIdx.x >> 5);
    grid_dep_wait();
    grid_dep_launch();
    if (m >= b.M) return;
    const TokenPlace at = token_place(b, m, lane);
    if (at.seq < 0) return;
    const int page = cache_page(b, at.seq, at.pos), off = at.pos & (b.page - 1);
    const int r = off & (REC_ROWS - 1), g = lane >> 3, c = lane & 7;
    uint4 raw[4];
    uint32_t sz[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool isv = i >= KV_H;
        const int h = i & 1;
        raw[i] = make_uint4(0u, 0u, 0u, 0u);
        sz[i] = 0;
        if (page < 0 || (isv ? v_out : k_out) == nullptr) continue;
        if (!Q4) {
            raw[i] = *(reinterpret_cast<const uint4 *>(static_cast<const bf16 *>(isv ? cv : ck) + row_bf16(b, page, h, off)) + lane);
        } else {
            const unsigned char *rec = static_cast<const unsigned char *>(ck) + record_of(b, page, h, off);
            raw[i].x = *reinterpret_cast<const uint32_t *>(rec + (isv ? REC_V : 0u) + r * 128 + c * 16 + g * 4);
            sz[i] = *reinterpret_cast<const uint32_t *>(rec + (isv ? REC_VSZ : REC_KSZ) + r * 16 + g * 4);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        TO *out = i >= KV_H ? v_out : k_out;
        if (out == nullptr) continue;
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        const float s = __uint_as_float(sz[i] << 16), z = __uint_as_float(sz[i] & 0xFFFF0000u);
        float x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            x[k] = Q4 ? fmaf(s, (float)((w[0] >> (4 * k)) & 15u), z)
                      : __uint_as_float((k & 1) ? (w[k >> 1] & 0xFFFF0000u) : (w[k >> 1] << 16));
        store8(out + ((size_t)m * KV_H + (i & 1)) * KV_D + 8 * lane, x);
    }
}

template <typename TO, bool Q4>
static cudaError_t launch_gather(const PagedBatch &b, const gdn_kv_cache *c, void *k_out, void *v_out, cudaStream_t s)
{
    const dim3 grid((unsigned)((b.M + KV_WARPS - 1) / KV_WARPS));
    return launch_pdl(kv_gather_kernel<TO, Q4>, grid, dim3(KV_WARPS * 32), 0, s, b, c->k, c->v, (TO *)k_out, (TO *)v_out);
}

cudaError_t launch_kv_gather(const gdn_paged_batch *b, const gdn_kv_cache *c, void *k_out, void *v_out,
                             gdn_dtype out_dt, cudaStream_t s)
{
    const PagedBatch pb = paged_batch(*b, *c);
    if (c->format == GDN_KV_Q4)
        return out_dt == GDN_F32 ? launch_gather<float, true>(pb, c, k_out, v_out, s) : launch_gather<bf16, true>(pb, c, k_out, v_out, s);
    return out_dt == GDN_F32 ? launch_gather<float, false>(pb, c, k_out, v_out, s) : launch_gather<bf16, false>(pb, c, k_out, v_out, s);
}

}  // namespace gdn
