// gdn_layer.cuh -- what the kernels around the mixers share (residual + norm,
// linear products, the mixture-of-experts layer): 8-element vector accesses
// and tensor maps of row-major bf16 matrices with any row stride.
#pragma once

#include <cuda.h>

#include "gdn_async.cuh"
#include "gdn_common.cuh"

namespace gdn {

constexpr int LD = GDN_HIDDEN;           // 2048: width of the residual stream

__device__ __forceinline__ void unpack8(uint4 u, float (&x)[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16));
}
// 8 consecutive elements, 16-byte aligned. Plain loads: an output may be its own input.
__device__ __forceinline__ void ld8(const float *p, float (&x)[8])
{
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void ld8(const bf16 *p, float (&x)[8]) { unpack8(*reinterpret_cast<const uint4 *>(p), x); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void st8(float *p, const float (&x)[8])
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void st8(bf16 *p, const float (&x)[8])
{
    *reinterpret_cast<uint4 *>(p) =
        make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// Whether the CTA has given up, one answer for the whole warp: another warp may set the flag
// between two lanes' reads, and lanes that disagree must not come to a step that all take together.
__device__ __forceinline__ bool warp_gave_up(const volatile int &aborted) { return __any_sync(0xffffffffu, aborted != 0); }

// Row-major bf16 matrix [rows][cols], row_stride elements from row to row (a
// multiple of 8), read in boxes of 64 columns x box_rows rows in the 128-byte
// swizzle; elements past either end read as zero. False if the driver's encoder
// is unavailable or rejects the arguments.
bool make_bf16_strided_map(CUtensorMap *map, const void *base, long long rows, int cols, long long row_stride,
                           int box_rows);

int sm_count();

}  // namespace gdn
