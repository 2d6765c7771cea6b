// gdn_paged_q4.cu -- attention of single tokens over the 4-bit paged cache.
//
// Bound by HBM: 288 bytes per cached position and KV head. At the measured copy
// rate an SM receives a 16-position record (4608 bytes) every 190 cycles, so
// what the codes cost on chip decides: expanding them to bf16 in shared memory
// for the 5th-generation tensor cores would write and read back 16 KiB per
// record, more than the shared-memory port carries in that time (128 bytes per
// cycle). So the codes go from shared memory to registers once and enter warp
// matrix instructions (m16n8k16, 8 query heads as N) as they are: nibble c in
// the low mantissa bits of 0x4300 is the bf16 number 128 + c, one logic
// operation per two codes. Steps and zeros stay out of the products:
//   q . k = sum_g s_g (sum_{d in g} q_d (128 + c_d)) + (z_g - 128 s_g) sum_{d in g} q_d,
//   o_d   = sum_p w'_p (128 + c_d) + sum_p (w_p z_p - 128 w'_p),  w'_p = bf16(w_p s_p),
// with the sums per group g of 64 dims in fp32. The one rounding to fewer bits is
// w'. Products with 128 + c lose nothing that matters: the 128s are taken out
// with the rounded w' they went in with.
//
// Work: gdn_paged.cuh with one token per item. A unit is 8 records, one per warp:
// each of the 8 warps runs its own online softmax over its records, and the warps
// meet once per piece. A ninth warp issues the copies, lane k for warp k: a
// record's 32 code rows as one tiled TMA box in the 128-byte swizzle (which makes
// every operand read below free of bank conflicts) and its steps and zeros as
// another, through a ring of four records per warp.
#include "gdn_paged.cuh"

namespace gdn {

__device__ unsigned int g_paged_q4_error;         // GDN_ERR_TIMEOUT if a bounded wait gave up

constexpr int DQ_WARPS = 8;
constexpr int DQ_THREADS = 32 * (DQ_WARPS + 1);
constexpr int DQ_STAGES = 4;
constexpr uint32_t DQ_CODES = 4096, DQ_SZ = 512;  // bytes of a record's codes; of its steps and zeros
constexpr int DQ_OSTRIDE = KV_D + 8;              // floats per head of a warp's output in shared memory
constexpr uint32_t DQ_RING = 0;
constexpr uint32_t DQ_RING_SZ = DQ_WARPS * DQ_STAGES * DQ_CODES;
constexpr uint32_t DQ_OUT = DQ_RING_SZ + DQ_WARPS * DQ_STAGES * DQ_SZ;
constexpr uint32_t DQ_SMALL = DQ_OUT + DQ_WARPS * KV_G * DQ_OSTRIDE * 4;

struct DqSmall {
    uint64_t full[DQ_WARPS][DQ_STAGES], empty[DQ_WARPS][DQ_STAGES];
    long long scan[DQ_THREADS / 32 + 1];
    PagedStart start;
    float ml[DQ_WARPS][KV_G][2];
    int abort;                                    // a wait gave up
    int stop;                                     // set by consumers before the barrier that all of them read it behind
};
constexpr size_t DQ_SMEM = DQ_SMALL + sizeof(DqSmall) + 1024;
static_assert(DQ_SMEM <= 232448, "shared memory of one CTA");

__device__ __forceinline__ void mma_m16n8k16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 8 x 8 transpose of 16-bit elements across the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// Codes t and t + 4 of a word as the bf16 pair (128 + c_t, 128 + c_{t+4}).
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int t) { return ((w >> (4 * t)) & 0x000F000Fu) | 0x43004300u; }

__device__ __forceinline__ float sz_step(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float sz_zero(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t word_of(const uint4 &v, int g) { return g == 0 ? v.x : g == 1 ? v.y : g == 2 ? v.z : v.w; }
__device__ __forceinline__ uint4 lds128(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

template <typename TO>
__global__ void __launch_bounds__(DQ_THREADS, 1) attn_paged_q4_kernel(const __grid_constant__ CUtensorMap cmap,
                                                                      const __grid_constant__ CUtensorMap smap,
                                                                      const PagedArgs a)
{
    extern __shared__ unsigned char smem_raw[];
    unsigned char *blk = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    DqSmall &ss = *reinterpret_cast<DqSmall *>(blk + DQ_SMALL);
    const uint32_t sb = smem_u32(blk);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const PagedBatch &b = a.b;

    if (tid < DQ_WARPS * DQ_STAGES) {
        mbar_init(smem_u32(&ss.full[0][0] + tid), 1);
        mbar_init(smem_u32(&ss.empty[0][0] + tid), 32);
    }
    if (tid == 0) ss.abort = ss.stop = 0;
    fence_mbar_init();
    grid_dep_wait();
    grid_dep_launch();
    find_start<DQ_THREADS>(a, blockIdx.x, ss.scan, &ss.start);   // ends in a CTA barrier
    const PagedStart st = ss.start;
    if (tid == 0) a.start[blockIdx.x] = st;
    const long long count = range_begin(st, blockIdx.x + 1, a.ranges) - range_begin(st, blockIdx.x, a.ranges);
    PieceWalk w;
    if (count > 0) w.begin(a, st, count);
    if (count == 0 || w.len == 0) return;
    const volatile int &aborted = ss.abort;
    auto codes_at = [&](int wp, uint32_t i) { return sb + DQ_RING + (wp * DQ_STAGES + i % DQ_STAGES) * DQ_CODES; };
    auto sz_at = [&](int wp, uint32_t i) { return sb + DQ_RING_SZ + (wp * DQ_STAGES + i % DQ_STAGES) * DQ_SZ; };

    if (warp == DQ_WARPS) {
        // ---- producer: lane k feeds warp k
        UnitWalk u;
        u.w = w;
        u.j = 0;
        const int recs = (b.num_pages * KV_H) << b.page_log2 >> 4;
        // this lane's record of the walk's unit: -1 if the item does not see it, past the end for a bad page
        auto record = [&]() {
            const int p = (u.w.unit + u.j) * PG_TILE + 16 * lane;
            if (lane >= DQ_WARPS || p >= tile_sees(a, u.w.t, u.w.tile)) return -1;
            const int page = cache_page(b, u.w.seq, p);
            return page < 0 ? recs : ((((page * KV_H + u.w.head) << b.page_log2) + (p & (b.page - 1))) >> 4);
        };
        uint32_t i = 0;
        bool ok = true;
        int rec = record();
        for (;;) {
            const bool more = !u.last(a);
            int next = -1;
            if (more) {                            // the next unit's page is looked up before this one waits
                u.next(a);
                next = record();
            }
            if (rec >= 0 && ok) {
                if (i >= DQ_STAGES)
                    ok = mbar_wait_bounded(smem_u32(&ss.empty[lane][i % DQ_STAGES]), (i / DQ_STAGES - 1) & 1);
                if (ok) {
                    const uint32_t bar = smem_u32(&ss.full[lane][i % DQ_STAGES]);
                    mbar_arrive_expect_tx(bar, DQ_CODES + DQ_SZ);
                    tma_load_3d(codes_at(lane, i), &cmap, 0, 0, rec, bar);
                    tma_load_2d(sz_at(lane, i), &smap, 0, rec, bar);
                    ++i;
                }
            }
            ok = __all_sync(0xffffffffu, ok && !aborted);
            if (!more || !ok) break;
            rec = next;
        }
        if (!ok) {                                 // copies in flight land before the CTA exits
            ss.abort = 1;
            if (lane < DQ_WARPS)
                for (uint32_t k = i > DQ_STAGES ? i - DQ_STAGES : 0; k < i; ++k)
                    mbar_wait_bounded(smem_u32(&ss.full[lane][k % DQ_STAGES]), (k / DQ_STAGES) & 1);
        }
    } else {
        // ---- consumers. Fragment coordinates: i = lane / 4, j = lane % 4.
        const int i4 = lane >> 2, j4 = lane & 3;
        uint32_t n = 0;                            // records consumed
        bool ok = true;
        for (;;) {
            const int sees = tile_sees(a, w.t, w.tile);
            const int mrow = w.t.row0 + w.tile;
            // Q^T operand: head i, dims of chunks 2 j and 2 j + 1 of each group, paired as code_pair
            // pairs the codes; and the sums of q over each group for heads 2 j, 2 j + 1
            uint32_t qf[4][2][4];
            float qs[4][2];
            {
                const bf16 *q = a.q + ((size_t)mrow * KV_HQ + KV_G * w.head + i4) * KV_D;
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    float sum = 0.0f;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(q + 64 * g + 8 * (2 * j4 + c)));
                        qf[g][c][0] = __byte_perm(v.x, v.z, 0x5410);   // dims 0, 4
                        qf[g][c][1] = __byte_perm(v.x, v.z, 0x7632);   // 1, 5
                        qf[g][c][2] = __byte_perm(v.y, v.w, 0x5410);   // 2, 6
                        qf[g][c][3] = __byte_perm(v.y, v.w, 0x7632);   // 3, 7
#pragma unroll
                        for (int k = 0; k < 4; ++k) sum += sz_step(word_of(v, k)) + sz_zero(word_of(v, k));
                    }
                    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                    qs[g][0] = __shfl_sync(0xffffffffu, sum, 8 * j4);
                    qs[g][1] = __shfl_sync(0xffffffffu, sum, 8 * j4 + 4);
                }
            }
            float o[4][4][4], bias[4][2], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                bias[g][0] = bias[g][1] = 0.0f;
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int k = 0; k < 4; ++k) o[g][t][k] = 0.0f;
            }
            for (int p0 = w.unit * PG_TILE + 16 * warp; p0 < min(sees, (w.unit + w.len) * PG_TILE); p0 += PG_TILE, ++n) {
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(&ss.full[warp][n % DQ_STAGES]), (n / DQ_STAGES) & 1));
                if (!ok) break;
                const uint32_t cb = codes_at(warp, n), zb = sz_at(warp, n);
                // scores of positions p0 + i and p0 + 8 + i for heads 2 j, 2 j + 1
                float s[4] = {0.f, 0.f, 0.f, 0.f};
                {
                    const uint32_t r0 = cb + i4 * 128, x0 = ((2 * j4) ^ i4) << 4, x1 = ((2 * j4 + 1) ^ i4) << 4;
                    const uint4 ka[2] = {lds128(r0 + x0), lds128(r0 + x1)};
                    const uint4 kb[2] = {lds128(r0 + 1024 + x0), lds128(r0 + 1024 + x1)};
                    uint4 z0 = lds128(zb + i4 * 16), z1 = lds128(zb + 128 + i4 * 16);
                    if (p0 + i4 >= sees) z0 = make_uint4(0u, 0u, 0u, 0u);        // rows past the context hold
                    if (p0 + 8 + i4 >= sees) z1 = make_uint4(0u, 0u, 0u, 0u);    // anything; codes are finite
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const uint32_t u = word_of(ka[c], g), v = word_of(kb[c], g);
                            mma_m16n8k16(acc, code_pair(u, 0), code_pair(v, 0), code_pair(u, 1), code_pair(v, 1),
                                         qf[g][c][0], qf[g][c][1]);
                            mma_m16n8k16(acc, code_pair(u, 2), code_pair(v, 2), code_pair(u, 3), code_pair(v, 3),
                                         qf[g][c][2], qf[g][c][3]);
                        }
                        const float s0 = sz_step(word_of(z0, g)), s1 = sz_step(word_of(z1, g));
                        const float t0 = fmaf(-128.0f, s0, sz_zero(word_of(z0, g))), t1 = fmaf(-128.0f, s1, sz_zero(word_of(z1, g)));
                        s[0] = fmaf(s0, acc[0], fmaf(t0, qs[g][0], s[0]));
                        s[1] = fmaf(s0, acc[1], fmaf(t0, qs[g][1], s[1]));
                        s[2] = fmaf(s1, acc[2], fmaf(t1, qs[g][0], s[2]));
                        s[3] = fmaf(s1, acc[3], fmaf(t1, qs[g][1], s[3]));
                    }
                    if (p0 + i4 >= sees) s[0] = s[1] = -INFINITY;
                    if (p0 + 8 + i4 >= sees) s[2] = s[3] = -INFINITY;
                }
                const float t0 = fmaxf(s[0], s[2]), t1 = fmaxf(s[1], s[3]);
                if (__any_sync(0xffffffffu, (t0 - m[0]) * SCORE_SCALE > RESCALE_AT || (t1 - m[1]) * SCORE_SCALE > RESCALE_AT)) {
                    // the references move to the maxima of all lanes that share a head
                    float x[2] = {fmaxf(t0, m[0]), fmaxf(t1, m[1])}, f[2];
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) {
                        x[0] = fmaxf(x[0], __shfl_xor_sync(0xffffffffu, x[0], d));
                        x[1] = fmaxf(x[1], __shfl_xor_sync(0xffffffffu, x[1], d));
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        f[k] = m[k] == -INFINITY ? 0.0f : ex2((m[k] - x[k]) * SCORE_SCALE);
                        m[k] = x[k];
                        l[k] *= f[k];
                    }
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        bias[g][0] *= f[0];
                        bias[g][1] *= f[1];
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            o[g][t][0] *= f[0];
                            o[g][t][1] *= f[1];
                            o[g][t][2] *= f[0];
                            o[g][t][3] *= f[1];
                        }
                    }
                }
                const float m0 = m[0] == -INFINITY ? 0.0f : m[0] * SCORE_SCALE, m1 = m[1] == -INFINITY ? 0.0f : m[1] * SCORE_SCALE;
                const float p[4] = {ex2(fmaf(s[0], SCORE_SCALE, -m0)), ex2(fmaf(s[1], SCORE_SCALE, -m1)),
                                    ex2(fmaf(s[2], SCORE_SCALE, -m0)), ex2(fmaf(s[3], SCORE_SCALE, -m1))};
                l[0] += p[0] + p[2];
                l[1] += p[1] + p[3];
                {
                    // V^T operand: dims on rows, so words of two positions are interleaved by halves
                    const uint32_t va = cb + 2048 + 2 * j4 * 128, x0 = (i4 ^ (2 * j4)) << 4, x1 = (i4 ^ (2 * j4 + 1)) << 4;
                    const uint4 v0 = lds128(va + x0), v1 = lds128(va + 128 + x1);
                    const uint4 v2 = lds128(va + 1024 + x0), v3 = lds128(va + 1152 + x1);
                    uint4 z0 = lds128(zb + 256 + i4 * 16), z1 = lds128(zb + 384 + i4 * 16);
                    if (p0 + i4 >= sees) z0 = make_uint4(0u, 0u, 0u, 0u);
                    if (p0 + 8 + i4 >= sees) z1 = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const float s0 = sz_step(word_of(z0, g)), s1 = sz_step(word_of(z1, g));
                        const uint32_t w0 = pack_bf16(p[0] * s0, p[1] * s0), w1 = pack_bf16(p[2] * s1, p[3] * s1);
                        const float e0 = sz_zero(word_of(z0, g)), e1 = sz_zero(word_of(z1, g));
                        bias[g][0] += fmaf(p[0], e0, p[2] * e1) - 128.0f * (sz_step(w0) + sz_step(w1));
                        bias[g][1] += fmaf(p[1], e0, p[3] * e1) - 128.0f * (sz_zero(w0) + sz_zero(w1));
                        const uint32_t b0 = transpose8(w0), b1 = transpose8(w1);
                        const uint32_t lo = __byte_perm(word_of(v0, g), word_of(v1, g), 0x5410), hi = __byte_perm(word_of(v0, g), word_of(v1, g), 0x7632);
                        const uint32_t lo2 = __byte_perm(word_of(v2, g), word_of(v3, g), 0x5410), hi2 = __byte_perm(word_of(v2, g), word_of(v3, g), 0x7632);
                        // product t: rows 0-7 are dims 8 i + 2 t of the group, rows 8-15 dims 8 i + 2 t + 1
                        mma_m16n8k16(o[g][0], code_pair(lo, 0), code_pair(lo, 1), code_pair(lo2, 0), code_pair(lo2, 1), b0, b1);
                        mma_m16n8k16(o[g][1], code_pair(lo, 2), code_pair(lo, 3), code_pair(lo2, 2), code_pair(lo2, 3), b0, b1);
                        mma_m16n8k16(o[g][2], code_pair(hi, 0), code_pair(hi, 1), code_pair(hi2, 0), code_pair(hi2, 1), b0, b1);
                        mma_m16n8k16(o[g][3], code_pair(hi, 2), code_pair(hi, 3), code_pair(hi2, 2), code_pair(hi2, 3), b0, b1);
                    }
                }
                mbar_arrive(smem_u32(&ss.empty[warp][n % DQ_STAGES]));
            }
            // the warps' outputs, maxima and sums meet in shared memory
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    l[k] += __shfl_xor_sync(0xffffffffu, l[k], d);
#pragma unroll
                    for (int g = 0; g < 4; ++g) bias[g][k] += __shfl_xor_sync(0xffffffffu, bias[g][k], d);
                }
            }
            float *os = reinterpret_cast<float *>(blk + DQ_OUT) + warp * KV_G * DQ_OSTRIDE;
#pragma unroll
            for (int g = 0; g < 4; ++g)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float4 *dst = reinterpret_cast<float4 *>(os + (2 * j4 + k) * DQ_OSTRIDE + 64 * g + 8 * i4);
                    dst[0] = make_float4(o[g][0][k] + bias[g][k], o[g][0][2 + k] + bias[g][k], o[g][1][k] + bias[g][k], o[g][1][2 + k] + bias[g][k]);
                    dst[1] = make_float4(o[g][2][k] + bias[g][k], o[g][2][2 + k] + bias[g][k], o[g][3][k] + bias[g][k], o[g][3][2 + k] + bias[g][k]);
                }
            if (i4 == 0)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    ss.ml[warp][2 * j4 + k][0] = m[k] * SCORE_SCALE;
                    ss.ml[warp][2 * j4 + k][1] = l[k];
                }
            if (!ok) ss.abort = ss.stop = 1;
            asm volatile("bar.sync 1, 256;" ::: "memory");
            {
                const int h = warp, d = 8 * lane;
                float M = -INFINITY, L = 0.0f, e[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < DQ_WARPS; ++k) M = fmaxf(M, ss.ml[k][h][0]);
                const float *src = reinterpret_cast<const float *>(blk + DQ_OUT) + h * DQ_OSTRIDE + d;
#pragma unroll 1
                for (int k = 0; k < DQ_WARPS; ++k) {
                    if (ss.ml[k][h][1] == 0.0f) continue;      // no records of this piece
                    const float f = ex2(ss.ml[k][h][0] - M);
                    const float4 x = *reinterpret_cast<const float4 *>(src + k * KV_G * DQ_OSTRIDE);
                    const float4 y = *reinterpret_cast<const float4 *>(src + k * KV_G * DQ_OSTRIDE + 4);
                    L += f * ss.ml[k][h][1];
                    e[0] += f * x.x; e[1] += f * x.y; e[2] += f * x.z; e[3] += f * x.w;
                    e[4] += f * y.x; e[5] += f * y.y; e[6] += f * y.z; e[7] += f * y.w;
                }
                if (w.whole()) {
                    finish8<TO>(a, mrow, KV_G * w.head + h, d, e, L != 0.0f ? 1.0f / L : 0.0f);
                } else {
                    const size_t slot = ((size_t)2 * blockIdx.x + (w.first ? 0 : 1)) * a.rows + h;
                    store8_out(a.part_o + slot * KV_D + d, e);
                    if (lane == 0) *reinterpret_cast<float2 *>(a.part_ml + slot * 2) = make_float2(M, L);
                }
            }
            const bool stop = *const_cast<const volatile int *>(&ss.stop) != 0;
            asm volatile("bar.sync 1, 256;" ::: "memory");
            if (stop || !w.more(a)) break;
            w.next(a);
        }
    }
    if (lane == 0 && ss.abort) atomicExch(&g_paged_q4_error, (unsigned int)GDN_ERR_TIMEOUT);
}

template <typename TO>
static cudaError_t launch_typed(const CUtensorMap &cm, const CUtensorMap &sm, const PagedArgs &a, cudaStream_t s)
{
    const cudaError_t e = smem_attr_once<attn_paged_q4_kernel<TO>>(DQ_SMEM);
    if (e != cudaSuccess) return e;
    return launch_pdl(attn_paged_q4_kernel<TO>, dim3(a.ranges), dim3(DQ_THREADS), DQ_SMEM, s, cm, sm, a);
}

cudaError_t launch_paged_q4(const PagedArgs &a, gdn_dtype out_dt, cudaStream_t s)
{
    // records as [n][32 rows][128 bytes] of codes, and [n][128 words] of steps and zeros; past the last: zeros
    CUtensorMap cm, sm;
    const cuuint64_t n = ((cuuint64_t)a.b.num_pages * KV_H << a.b.page_log2) / REC_ROWS;
    const cuuint64_t cd[3] = {128, 2 * REC_ROWS, n}, cs[2] = {128, REC_BYTES}, sd[2] = {DQ_SZ / 4, n}, sst[1] = {REC_BYTES};
    const cuuint32_t cbox[3] = {128, 2 * REC_ROWS, 1}, sbox[2] = {DQ_SZ / 4, 1};
    if (!encode_tiled(&cm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, a.ck, cd, cs, cbox, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tiled(&sm, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, static_cast<const char *>(a.ck) + REC_KSZ, sd, sst, sbox,
                      CU_TENSOR_MAP_SWIZZLE_NONE))
        return cudaErrorInvalidValue;
    return out_dt == GDN_F32 ? launch_typed<float>(cm, sm, a, s) : launch_typed<bf16>(cm, sm, a, s);
}

// Device address of this file's error word, for gdn_device_error.
void *paged_q4_error_word()
{
    void *p = nullptr;
    return cudaGetSymbolAddress(&p, g_paged_q4_error) == cudaSuccess ? p : nullptr;
}

}  // namespace gdn
