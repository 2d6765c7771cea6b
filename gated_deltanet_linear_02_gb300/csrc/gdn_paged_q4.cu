// gdn_paged_q4.cu -- attention of single tokens over the 4-bit paged cache.
//
// 288 bytes per cached position and KV head: 256 contexts of up to 4,096 take 109 us
// (4.2 TB/s, 62% of a copy's rate), bound by the instructions per record (about 580)
// and their latency rather than by HBM. At the measured copy
// rate an SM receives a 16-position record (4608 bytes) every 190 cycles, so
// what the codes cost on chip decides: expanding them to bf16 in shared memory
// for the 5th-generation tensor cores would write and read back 16 KiB per
// record, more than the shared-memory port carries in that time (128 bytes per
// cycle). So the codes go from shared memory to registers once and enter warp
// matrix instructions (m16n8k16, 8 query heads as N) almost as they are, one logic
// operation per two codes and few shifts:
//  - keys in fp16: nibble c in bits 0-3 of 0x6400 is 1024 + c, in bits 4-7 1024 +
//    16 c, so a word of eight codes needs one shift; q enters in fp16, scaled by a
//    power of two per head (exact down to 2^-20 of the head's largest element) and
//    by 1/16 where the code has its 16;
//  - values in bf16: the sum runs over positions, so words of two positions are
//    interleaved by halves, and nibble c in the low bits of 0x4300 is 128 + c, and
//    inverted in those of 0xC300 c - 143: the positions of a record take these in
//    turn, odd ones first in its second half.
// (fp8 instructions would take the nibbles as they are, 0..15 being c 2^-9 in e4m3,
// but they are carried out as conversions to fp16 here: measured 10% slower.)
// Steps and zeros stay out of the products: with sums per group g of 64 dims,
//   q . k = sum_g s_g (sum_{d in g} q_d (1024 + c_d) - 1024 sum q_d) + z_g sum_{d in g} q_d,
//   o_d   = sum_p w'_p (128 + c_d, or c_d - 143) + sum_p (w_p (z_p + 8 s_p) - 136 w'_p, or + 135 w'_p),
//   w'_p  = bf16(w_p s_p).
// The roundings to fewer bits are w' and q's elements below 2^-20 of the largest.
// The offsets are taken out with the rounded numbers they went in with; the 8 puts
// the rounding of w' on c - 8, half as large as c.
// The warp instructions' sums are truncated, so a sum that an offset makes large
// moves by a part of that offset, always in one direction. So positions next to
// each other, and the halves, carry offsets of opposite sign, and every DQ_FOLD
// records a warp takes what they have left out of its sums. Error against 64 bits
// (norm of the difference over that of the result, values about zero, fp32 outputs):
// 1.6e-3 to 1.8e-3 from 1,024 to 262,144 positions in one piece, the rounding of w'
// alone; with 128 + c throughout and one correction at the end 1.8e-3 at 4,096, 8e-3
// at 16,384, 0.13 at 65,536. The keys' 1,024 q are gone after each 64 dims of a
// record: below 1e-4 of the spread of a score.
//
// Work: gdn_paged.cuh with one token per item. The records of a piece go round the
// 11 warps, each with its own online softmax, and the warps meet once per piece.
// A twelfth warp issues the copies, lane k for warp k: a
// record's 32 code rows as one tiled TMA box in the 128-byte swizzle (which makes
// every operand read below free of bank conflicts) and its steps and zeros as
// another, through a ring of three records per warp.
#include <cuda_fp16.h>

#include <type_traits>

#include "gdn_paged.cuh"

namespace gdn {

__device__ unsigned int g_paged_q4_error;         // GDN_ERR_TIMEOUT if a bounded wait gave up

constexpr int DQ_WARPS = 11;                      // with the producer three warps per scheduler, 168 registers each
constexpr int DQ_THREADS = 32 * (DQ_WARPS + 1);
constexpr int DQ_STAGES = 3;
constexpr uint32_t DQ_CODES = 4096, DQ_SZ = 512;  // bytes of a record's codes; of its steps and zeros
// Records of a warp after which the offsets leave its sums. A decode batch takes 109.0 us with 32, 109.8 with 16,
// 110.5 with 8 (108.5 when they leave at the end only); where one of every 16 positions has all the weight, so that
// offsets do not cancel, 262,144 positions in a piece give an error of 2.1e-3, 1.8e-3, 1.7e-3.
constexpr int DQ_FOLD = 32;
constexpr int DQ_OSTRIDE = KV_D + 8;              // floats per head of a warp's output in shared memory
constexpr uint32_t DQ_RING = 0;
constexpr uint32_t DQ_RING_SZ = DQ_WARPS * DQ_STAGES * DQ_CODES;
constexpr uint32_t DQ_OUT = DQ_RING_SZ + DQ_WARPS * DQ_STAGES * DQ_SZ;
constexpr uint32_t DQ_SMALL = DQ_OUT + DQ_WARPS * (KV_G / 2) * DQ_OSTRIDE * 4;

// A piece's queries as its warps take them, made by the producer warp.
struct DqQuery {
    uint4 frag[8][32];                            // [2 g + c][lane]: B operands of the key products
    float4 aux[4][4];                             // [g][j]: what the 1024s add, negated, and the sums of q, for heads 2 j, 2 j + 1
    float2 back[4];                               // [j]: the scale back
};
constexpr int DQ_QUERIES = 4;                     // short pieces run up to three ahead

struct DqSmall {
    DqQuery query[DQ_QUERIES];
    uint64_t q_full[DQ_QUERIES], q_empty[DQ_QUERIES];
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
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with fp16 operands; mma_f16_from starts from the accumulator (c0, c1, c0, c1).
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_from(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1, float c0, float c1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%10,%11};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}
// 8 x 8 transpose of 16-bit elements across the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// (w & mask) | magic in one logic operation; the masks are kept in registers.
__device__ __forceinline__ uint32_t mask_or(uint32_t w, uint32_t mask, uint32_t magic)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(magic));
    return r;
}
// (w & mask) ^ magic: halves of 0x4300 give 128 + c, halves of 0xC30F the negative of 128 + (15 - c), c - 143.
__device__ __forceinline__ uint32_t mask_xor(uint32_t w, uint32_t mask, uint32_t magic)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(r) : "r"(w), "r"(mask), "r"(magic));
    return r;
}
__device__ __forceinline__ float sz_step(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float sz_zero(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t word_of(const uint4 &v, int g) { return g == 0 ? v.x : g == 1 ? v.y : g == 2 ? v.z : v.w; }
__device__ __forceinline__ uint4 lds128(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

// Queries of one item into shared memory, by one warp with the fragment coordinates
// i = lane / 4, j = lane % 4. B operand of the key products: head i, dims of chunks
// 2 j and 2 j + 1 of each group, in fp16, scaled by a power of two per head that
// brings its largest element to 128..256, and by 1/16 more where the code has its
// 16; paired as the codes unpack: (0, 4), (1, 5) / 16, (2, 6), (3, 7) / 16.
__device__ __noinline__ void make_query(const uint4 *q, DqQuery &out, int lane)
{
    const int j4 = lane & 3;
    uint32_t qf[4][2][4];
    float qs[4][2], top = 0.0f;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        float sum = 0.0f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const uint4 v = q[8 * g + c];          // not __ldg: the kernel before may have written them while this one started
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                qf[g][c][k] = word_of(v, k);
                sum += sz_step(word_of(v, k)) + sz_zero(word_of(v, k));
                top = fmaxf(top, fmaxf(fabsf(sz_step(word_of(v, k))), fabsf(sz_zero(word_of(v, k)))));
            }
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        qs[g][0] = __shfl_sync(0xffffffffu, sum, 8 * j4);
        qs[g][1] = __shfl_sync(0xffffffffu, sum, 8 * j4 + 4);
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int ex = min(max((int)(__float_as_uint(top) >> 23), 24), 253);   // top in [2^(ex-127), 2^(ex-126))
    const float up = __uint_as_float((uint32_t)(261 - ex) << 23);         // 2^(134 - ex)
    const float down = __uint_as_float((uint32_t)(ex - 7) << 23);          // 2^(ex - 134)
    const float back0 = __shfl_sync(0xffffffffu, down, 8 * j4), back1 = __shfl_sync(0xffffffffu, down, 8 * j4 + 4);
    if (lane < 4) out.back[lane] = make_float2(back0, back1);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        float sum = 0.0f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float d[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                d[2 * k] = sz_step(qf[g][c][k]) * up;
                d[2 * k + 1] = sz_zero(qf[g][c][k]) * (up * 0.0625f);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const __half2 h = __floats2half2_rn(d[k], d[k + 4]);
                qf[g][c][k] = *reinterpret_cast<const uint32_t *>(&h);
                const float2 f = __half22float2(h);
                sum += f.x + f.y;
            }
        }
        sum *= -1024.0f;
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        const float off0 = __shfl_sync(0xffffffffu, sum, 8 * j4), off1 = __shfl_sync(0xffffffffu, sum, 8 * j4 + 4);
        if (lane < 4) out.aux[g][lane] = make_float4(off0, off1, qs[g][0], qs[g][1]);
#pragma unroll
        for (int c = 0; c < 2; ++c) out.frag[2 * g + c][lane] = make_uint4(qf[g][c][0], qf[g][c][1], qf[g][c][2], qf[g][c][3]);
    }
}

__device__ __forceinline__ void consumer_bar() { asm volatile("bar.sync 1, %0;" ::"n"(32 * DQ_WARPS) : "memory"); }

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
    if (tid < DQ_QUERIES) {
        mbar_init(smem_u32(&ss.q_full[tid]), 32);
        mbar_init(smem_u32(&ss.q_empty[tid]), DQ_WARPS);
    }
    if (tid == 0) ss.abort = ss.stop = 0;
    fence_mbar_init();
    grid_dep_wait();
    grid_dep_launch();
    find_start<DQ_THREADS>(a, blockIdx.x, ss.scan, &ss.start);   // ends in a CTA barrier
    const PagedStart st = ss.start;
    if (tid == 0) a.start[blockIdx.x] = st;
    const long long count = range_begin(st, blockIdx.x + 1) - range_begin(st, blockIdx.x);
    PieceWalk w;
    if (count > 0) w.begin(a, st, count);
    if (count == 0 || w.len == 0) return;
    const volatile int &aborted = ss.abort;
    auto codes_at = [&](int wp, uint32_t i) { return sb + DQ_RING + (wp * DQ_STAGES + i) * DQ_CODES; };
    auto sz_at = [&](int wp, uint32_t i) { return sb + DQ_RING_SZ + (wp * DQ_STAGES + i) * DQ_SZ; };

    // a piece's queries into one of the buffers; a whole warp
    auto query = [&](uint32_t qb, int token, int head) {
        make_query(reinterpret_cast<const uint4 *>(a.q + ((size_t)token * KV_HQ + KV_G * head + (lane >> 2)) * KV_D) + 2 * (lane & 3),
                   ss.query[qb], lane);
        mbar_arrive(smem_u32(&ss.q_full[qb]));
    };
    // where the positions of a piece end
    auto piece_end = [&](const PieceWalk &p) { return min(tile_sees(a, p.t, p.tile), (p.unit + p.len) * PG_TILE); };

    if (warp == DQ_WARPS) {
        // ---- producer: lane k feeds warp k
        const int recs = (b.num_pages * KV_H) << b.page_log2 >> 4;
        int base = 0;                              // first record of the round, from the piece's first position
        bool more = true;
        // A round's record of this lane: whether it has one, its page table entry (a load that is two
        // rounds old when its value is first needed) and its place in the page; in a piece's first round
        // also the piece's token and head, else below 0.
        struct Rec {
            bool round, mine, whole;
            int page, in_page, token, head;
        };
        uint32_t piece = 0;
        bool ok = true;
        auto fetch = [&]() {
            Rec r = {more, false, w.whole(), 0, 0, base == 0 ? w.t.row0 + w.tile : -1, w.head};
            if (!more) return r;
            const int p = w.unit * PG_TILE + 16 * (base + lane), end = piece_end(w);
            if (lane < DQ_WARPS && p < end) {
                r.mine = true;
                r.page = __ldg(b.table + (size_t)w.seq * b.max_pages + (p >> b.page_log2));
                r.in_page = (w.head << b.page_log2) + (p & (b.page - 1));
            }
            base += DQ_WARPS;
            if (w.unit * PG_TILE + 16 * base >= end) {
                more = w.more(a);
                if (more) w.next(a);
                base = 0;
            }
            return r;
        };
        uint32_t i = 0;
        Rec r0 = fetch(), r1 = fetch();
        while (r0.round && ok) {
            const Rec r2 = fetch();
            if (r0.mine && ok) {
                if (i >= DQ_STAGES)
                    ok = mbar_wait_bounded(smem_u32(&ss.empty[lane][i % DQ_STAGES]), (i / DQ_STAGES - 1) & 1);
                if (ok) {
                    // a page id outside the cache reads past its end: zeros
                    const int rec = (unsigned)r0.page < (unsigned)b.num_pages
                                        ? (((r0.page * KV_H) << b.page_log2) + r0.in_page) >> 4 : recs;
                    const uint32_t bar = smem_u32(&ss.full[lane][i % DQ_STAGES]);
                    mbar_arrive_expect_tx(bar, DQ_CODES + DQ_SZ);
                    tma_load_3d(codes_at(lane, i % DQ_STAGES), &cmap, 0, 0, rec, bar);
                    tma_load_2d(sz_at(lane, i % DQ_STAGES), &smap, 0, rec, bar);
                    ++i;
                }
            }
            ok = __all_sync(0xffffffffu, ok && !aborted);
            if (ok && r0.token >= 0) {             // the piece's queries, while its first records come (before them: 117 us)
                const uint32_t qb = piece % DQ_QUERIES;
                if (piece >= DQ_QUERIES)
                    ok = __all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(&ss.q_empty[qb]), (piece / DQ_QUERIES - 1) & 1));
                if (ok) {
                    if (piece > 0) query(qb, r0.token, r0.head);   // warp 0 makes the first
                    ++piece;
                    if (a.gate != nullptr && r0.whole) // and its gates, for the epilogue: 128 bytes per lane
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.gate + r0.token * a.gate_row + (KV_G * r0.head + (lane >> 2)) * a.gate_head + 64 * (lane & 3)));
                }
            }
            if (!ok) break;
            r0 = r1;
            r1 = r2;
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
        uint32_t slot = 0, phase = 0, piece = 0;   // of the warp's ring; pieces begun
        uint32_t mask, plus_minus, minus_plus, mask16, one;   // not constants to the compiler, so that they stay in registers
        asm volatile("mov.u32 %0, 0x000F000F;\n\tmov.u32 %1, 0xC30F4300;\n\tmov.u32 %2, 0x4300C30F;" : "=r"(mask), "=r"(plus_minus), "=r"(minus_plus));
        asm volatile("mov.u32 %0, 0x00F000F0;\n\tmov.u32 %1, 0x64006400;" : "=r"(mask16), "=r"(one));
        // what takes the offset out, for positions i and 8 + i of a record
        const float back0 = i4 & 1 ? 135.0f : -136.0f, back1 = i4 & 1 ? -136.0f : 135.0f;
        bool ok = true;
        if (warp == 0) query(0, w.t.row0 + w.tile, w.head);
        for (;;) {
            const int sees = tile_sees(a, w.t, w.tile);
            const int mrow = w.t.row0 + w.tile;
            const uint32_t qb = piece % DQ_QUERIES;
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(&ss.q_full[qb]), (piece / DQ_QUERIES) & 1));
            ++piece;
            float o[4][4][4], bias[4][2], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                bias[g][0] = bias[g][1] = 0.0f;
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int k = 0; k < 4; ++k) o[g][t][k] = 0.0f;
            }
            const int end = piece_end(w);
            int folds = DQ_FOLD;                   // records until the biases next go into the outputs
            auto sum_bias = [&]() {                // over the lanes that share a head
#pragma unroll
                for (int d = 4; d < 32; d <<= 1)
#pragma unroll
                    for (int g = 0; g < 4; ++g)
#pragma unroll
                        for (int k = 0; k < 2; ++k) bias[g][k] += __shfl_xor_sync(0xffffffffu, bias[g][k], d);
            };
            for (int p0 = w.unit * PG_TILE + 16 * warp; p0 < end && ok; p0 += 16 * DQ_WARPS) {
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(&ss.full[warp][slot]), phase));
                if (!ok) break;
                const uint32_t cb = codes_at(warp, slot), zb = sz_at(warp, slot);
                auto record = [&](auto tail) {     // tail: the context ends inside the record
                // scores of positions p0 + i and p0 + 8 + i for heads 2 j, 2 j + 1
                float s[4] = {0.f, 0.f, 0.f, 0.f};
                {
                    const uint32_t r0 = cb + i4 * 128, x0 = ((2 * j4) ^ i4) << 4, x1 = ((2 * j4 + 1) ^ i4) << 4;
                    const uint4 ka[2] = {lds128(r0 + x0), lds128(r0 + x1)};
                    const uint4 kb[2] = {lds128(r0 + 1024 + x0), lds128(r0 + 1024 + x1)};
                    uint4 z0 = lds128(zb + i4 * 16), z1 = lds128(zb + 128 + i4 * 16);
                    if (tail.value) {              // rows past the context hold anything; codes are finite
                        if (p0 + i4 >= sees) z0 = make_uint4(0u, 0u, 0u, 0u);
                        if (p0 + 8 + i4 >= sees) z1 = make_uint4(0u, 0u, 0u, 0u);
                    }
                    float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        float acc[4];
                        const float4 aux = ss.query[qb].aux[g][j4];
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const uint32_t u = word_of(ka[c], g), v = word_of(kb[c], g);
                            const uint4 qf = ss.query[qb].frag[2 * g + c][lane];
                            const uint32_t x = u >> 8, y = v >> 8;
                            if (c == 0)
                                mma_f16_from(acc, mask_or(u, mask, one), mask_or(v, mask, one), mask_or(u, mask16, one),
                                             mask_or(v, mask16, one), qf.x, qf.y, aux.x, aux.y);
                            else
                                mma_f16(acc, mask_or(u, mask, one), mask_or(v, mask, one), mask_or(u, mask16, one),
                                        mask_or(v, mask16, one), qf.x, qf.y);
                            mma_f16(acc, mask_or(x, mask, one), mask_or(y, mask, one), mask_or(x, mask16, one),
                                    mask_or(y, mask16, one), qf.z, qf.w);
                        }
                        const float s0 = sz_step(word_of(z0, g)), s1 = sz_step(word_of(z1, g));
                        const float e0 = sz_zero(word_of(z0, g)), e1 = sz_zero(word_of(z1, g));
                        t[0] = fmaf(s0, acc[0], t[0]);
                        t[1] = fmaf(s0, acc[1], t[1]);
                        t[2] = fmaf(s1, acc[2], t[2]);
                        t[3] = fmaf(s1, acc[3], t[3]);
                        s[0] = fmaf(e0, aux.z, s[0]);
                        s[1] = fmaf(e0, aux.w, s[1]);
                        s[2] = fmaf(e1, aux.z, s[2]);
                        s[3] = fmaf(e1, aux.w, s[3]);
                    }
                    const float2 back = ss.query[qb].back[j4];
                    s[0] = fmaf(t[0], back.x, s[0]);
                    s[1] = fmaf(t[1], back.y, s[1]);
                    s[2] = fmaf(t[2], back.x, s[2]);
                    s[3] = fmaf(t[3], back.y, s[3]);
                    if (tail.value) {
                        if (p0 + i4 >= sees) s[0] = s[1] = -INFINITY;
                        if (p0 + 8 + i4 >= sees) s[2] = s[3] = -INFINITY;
                    }
                }
                // V^T operand: dims on rows, so words of two positions are interleaved by halves
                const uint32_t va = cb + 2048 + 2 * j4 * 128, x0 = (i4 ^ (2 * j4)) << 4, x1 = (i4 ^ (2 * j4 + 1)) << 4;
                const uint4 v0 = lds128(va + x0), v1 = lds128(va + 128 + x1);
                const uint4 v2 = lds128(va + 1024 + x0), v3 = lds128(va + 1152 + x1);
                uint4 z0 = lds128(zb + 256 + i4 * 16), z1 = lds128(zb + 384 + i4 * 16);
                if (tail.value) {
                    if (p0 + i4 >= sees) z0 = make_uint4(0u, 0u, 0u, 0u);
                    if (p0 + 8 + i4 >= sees) z1 = make_uint4(0u, 0u, 0u, 0u);
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
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const float s0 = sz_step(word_of(z0, g)), s1 = sz_step(word_of(z1, g));
                        const uint32_t w0 = pack_bf16(p[0] * s0, p[1] * s0), w1 = pack_bf16(p[2] * s1, p[3] * s1);
                        const float e0 = fmaf(8.0f, s0, sz_zero(word_of(z0, g))), e1 = fmaf(8.0f, s1, sz_zero(word_of(z1, g)));
                        bias[g][0] += fmaf(p[0], e0, p[2] * e1) + fmaf(back0, sz_step(w0), back1 * sz_step(w1));
                        bias[g][1] += fmaf(p[1], e0, p[3] * e1) + fmaf(back0, sz_zero(w0), back1 * sz_zero(w1));
                        const uint32_t b0 = transpose8(w0), b1 = transpose8(w1);
                        const uint32_t lo = __byte_perm(word_of(v0, g), word_of(v1, g), 0x5410), hi = __byte_perm(word_of(v0, g), word_of(v1, g), 0x7632);
                        const uint32_t lo2 = __byte_perm(word_of(v2, g), word_of(v3, g), 0x5410), hi2 = __byte_perm(word_of(v2, g), word_of(v3, g), 0x7632);
                        // product t: rows 0-7 are dims 8 i + 2 t of the group, rows 8-15 dims 8 i + 2 t + 1
                        mma_m16n8k16(o[g][0], mask_xor(lo, mask, plus_minus), mask_xor(lo >> 4, mask, plus_minus), mask_xor(lo2, mask, minus_plus), mask_xor(lo2 >> 4, mask, minus_plus), b0, b1);
                        mma_m16n8k16(o[g][1], mask_xor(lo >> 8, mask, plus_minus), mask_xor(lo >> 12, mask, plus_minus), mask_xor(lo2 >> 8, mask, minus_plus), mask_xor(lo2 >> 12, mask, minus_plus), b0, b1);
                        mma_m16n8k16(o[g][2], mask_xor(hi, mask, plus_minus), mask_xor(hi >> 4, mask, plus_minus), mask_xor(hi2, mask, minus_plus), mask_xor(hi2 >> 4, mask, minus_plus), b0, b1);
                        mma_m16n8k16(o[g][3], mask_xor(hi >> 8, mask, plus_minus), mask_xor(hi >> 12, mask, plus_minus), mask_xor(hi2 >> 8, mask, minus_plus), mask_xor(hi2 >> 12, mask, minus_plus), b0, b1);
                    }
                }
                };
                if (p0 + 16 > sees) record(std::true_type());
                else record(std::false_type());
                mbar_arrive(smem_u32(&ss.empty[warp][slot]));
                if (++slot == DQ_STAGES) {
                    slot = 0;
                    phase ^= 1;
                }
                if (--folds == 0) {                // the offsets out of the sums
                    folds = DQ_FOLD;
                    sum_bias();
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
#pragma unroll
                        for (int t = 0; t < 4; ++t)
#pragma unroll
                            for (int k = 0; k < 4; ++k) o[g][t][k] += bias[g][k & 1];
                        bias[g][0] = bias[g][1] = 0.0f;
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ss.q_empty[qb]));
            // the warps' outputs, maxima and sums meet in shared memory, four heads at a time
#pragma unroll
            for (int d = 4; d < 32; d <<= 1)
#pragma unroll
                for (int k = 0; k < 2; ++k) l[k] += __shfl_xor_sync(0xffffffffu, l[k], d);
            sum_bias();
            if (i4 == 0)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    ss.ml[warp][2 * j4 + k][0] = m[k] * SCORE_SCALE;
                    ss.ml[warp][2 * j4 + k][1] = l[k];
                }
            if (!ok) ss.abort = ss.stop = 1;
            float *const all = reinterpret_cast<float *>(blk + DQ_OUT);
            uint2 gates[2] = {};                   // of the warp's outputs in either half, before the warps wait for each other
            if (a.gate != nullptr && w.whole() && warp < 8)
#pragma unroll
                for (int half = 0; half < 2; ++half)
                    gates[half] = *(reinterpret_cast<const uint2 *>(a.gate + mrow * a.gate_row + (KV_G * w.head + 4 * half + (warp >> 1)) * a.gate_head) + 32 * (warp & 1) + lane);
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                if (j4 >> 1 == half) {
                    float *os = all + (warp * (KV_G / 2) + 2 * (j4 & 1)) * DQ_OSTRIDE + 8 * i4;
#pragma unroll
                    for (int g = 0; g < 4; ++g)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float4 *dst = reinterpret_cast<float4 *>(os + k * DQ_OSTRIDE + 64 * g);
                            dst[0] = make_float4(o[g][0][k] + bias[g][k], o[g][0][2 + k] + bias[g][k], o[g][1][k] + bias[g][k], o[g][1][2 + k] + bias[g][k]);
                            dst[1] = make_float4(o[g][2][k] + bias[g][k], o[g][2][2 + k] + bias[g][k], o[g][3][k] + bias[g][k], o[g][3][2 + k] + bias[g][k]);
                        }
                }
                consumer_bar();
                if (warp < 8) {                    // two warps per head, 4 dims per lane
                    const int hl = warp >> 1, h = 4 * half + hl, d = 128 * (warp & 1) + 4 * lane;
                    float M = -INFINITY, L = 0.0f;
                    float4 e = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int k = 0; k < DQ_WARPS; ++k) M = fmaxf(M, ss.ml[k][h][0]);
                    const float *src = all + hl * DQ_OSTRIDE + d;
#pragma unroll
                    for (int k = 0; k < DQ_WARPS; ++k) {
                        const float lk = ss.ml[k][h][1], f = lk != 0.0f ? ex2(ss.ml[k][h][0] - M) : 0.0f;   // 0: no records
                        const float4 x = *reinterpret_cast<const float4 *>(src + k * (KV_G / 2) * DQ_OSTRIDE);
                        L = fmaf(f, lk, L);
                        e.x = fmaf(f, x.x, e.x); e.y = fmaf(f, x.y, e.y); e.z = fmaf(f, x.z, e.z); e.w = fmaf(f, x.w, e.w);
                    }
                    if (w.whole()) {
                        finish4<TO>(a, half == 0 ? gates[0] : gates[1], mrow, KV_G * w.head + h, d, e, sees > 0 ? 1.0f / L : 0.0f);   // nothing seen: zeros
                    } else {
                        const size_t at = ((size_t)2 * blockIdx.x + (w.first ? 0 : 1)) * a.rows + h;
                        *reinterpret_cast<float4 *>(a.part_o + at * KV_D + d) = e;
                        if (lane == 0) *reinterpret_cast<float2 *>(a.part_ml + at * 2) = make_float2(M, L);
                    }
                }
                if (half == 0) consumer_bar();
            }
            const bool stop = *const_cast<const volatile int *>(&ss.stop) != 0;
            consumer_bar();
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
    return launch_pdl(attn_paged_q4_kernel<TO>, dim3(PG_RANGES), dim3(DQ_THREADS), DQ_SMEM, s, cm, sm, a);
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
