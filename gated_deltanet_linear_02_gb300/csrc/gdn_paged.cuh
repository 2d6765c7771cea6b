// gdn_paged.cuh -- how the paged attention kernels share out their work.
//
// An item is 16 consecutive new tokens of one sequence (the last one may have
// fewer), or a single token, and one KV head: up to 128 query rows (8 heads x 16
// tokens) that read the same keys and values. Its units are the 128-position tiles of the context
// that its last token sees, at least one. The units of all items, in order of
// sequence, tokens, head and position, are cut into one even range per CTA,
// wherever that falls: contexts of any mix of lengths and batches of any size
// keep every SM busy to the end. An item inside one CTA's range is finished
// there; the pieces of an item that spans CTAs go to the workspace as
// unnormalised outputs with their maximum and sum, at most two per CTA (its
// first and its last), and a second kernel joins them. Lengths are read on the
// device, so a captured call follows them from replay to replay.
#pragma once

#include <cuda.h>

#include <mutex>

#include "gdn_async.cuh"
#include "gdn_kv.cuh"
#include "gdn_tma.cuh"

namespace gdn {

constexpr int PG_TOK = 16;                        // tokens per item, at most
constexpr int PG_TILE = 128;                      // positions per unit
constexpr int PG_RANGES = 152;                    // one CTA per SM

constexpr float SCORE_SCALE = 1.4426950408889634f / 16.0f;   // log2 e / sqrt(256)
constexpr float RESCALE_AT = 8.0f;                // powers of two a maximum may pass the reference by

struct PagedArgs {
    PagedBatch b;
    const void *ck, *cv;
    const bf16 *q, *gate;
    long long gate_row, gate_head;
    void *out;
    struct PagedStart *start;                     // [PG_RANGES]
    float *part_o;                                // [2 * PG_RANGES][rows][256]
    float *part_ml;                               // [2 * PG_RANGES][rows][2]
    int rows;                                     // rows per piece in the workspace: 8 min(max_q, 16)
    int lead;                                     // leading steps of an item: its epilogue and start, counted in units
    int tok, tok_log2;                            // tokens per item: 16 or 1
};

// One sequence's new tokens: packed rows [row0, row0 + n) at positions first,
// first + 1, ...
struct SeqTokens {
    int row0, n, first;
};
// Where a range starts; the whole call has quot * PG_RANGES + rem steps.
struct PagedStart {
    long long quot;
    int rem;
    int seq, tile, head, step;
    SeqTokens t;                                  // of sequence seq
};

__device__ __forceinline__ SeqTokens seq_tokens(const PagedBatch &b, int s)
{
    SeqTokens t;
    const int ctx = __ldg(b.ctx + s);
    if (b.cu == nullptr) {
        t.row0 = s;
        t.n = 1;
    } else {
        t.row0 = min(max(__ldg(b.cu + s), 0), b.M);
        t.n = min(min(max(__ldg(b.cu + s + 1), t.row0), b.M) - t.row0, b.max_q);
    }
    // positions past 2^30 + 2^24 see what 2^30 sees; the clamp keeps sums in 32 bits
    t.first = (int)max(min((long long)ctx - t.n, 1ll << 30), -(1ll << 30));
    return t;
}

// Positions the last token of tile i sees, and the tile's units.
__device__ __forceinline__ int tile_sees(const PagedArgs &a, const SeqTokens &t, int i)
{
    return min(t.first + min((i + 1) << a.tok_log2, t.n), a.b.max_pages << a.b.page_log2);
}
__device__ __forceinline__ int tile_units(const PagedArgs &a, const SeqTokens &t, int i)
{
    return max((tile_sees(a, t, i) + PG_TILE - 1) / PG_TILE, 1);
}
__device__ __forceinline__ int seq_tiles(const PagedArgs &a, const SeqTokens &t) { return (t.n + a.tok - 1) >> a.tok_log2; }

// Units of tiles 0 .. i-1, per head. With x = floor((first + 127) / tok) and
// D = 128 / tok, whole tile j (from 1) has floor((x + j) / D) units, and the sum
// of floor(m / D) over m = 0 .. D q + r is D q (q - 1) / 2 + q (r + 1). Contexts
// that start below 0 or end past the table are summed term by term.
__device__ __forceinline__ long long units_before(const PagedArgs &a, const SeqTokens &t, int i)
{
    if (t.first < 0 || t.first + t.n > (a.b.max_pages << a.b.page_log2)) {
        long long u = 0;
        for (int j = 0; j < i; ++j) u += tile_units(a, t, j);
        return u;
    }
    const int tiles = seq_tiles(a, t), whole = min(i, t.n >> a.tok_log2), dl = 7 - a.tok_log2;
    auto sum = [dl](long long m) {
        const long long q = m >> dl;
        return ((q * (q - 1)) << dl >> 1) + q * ((m & ((1 << dl) - 1)) + 1);
    };
    const int x = (t.first + PG_TILE - 1) >> a.tok_log2;
    long long u = sum(x + whole) - sum(x);
    if (i == tiles && whole < tiles) u += tile_units(a, t, tiles - 1);
    return u;
}
// Steps of tiles 0 .. i-1, both heads.
__device__ __forceinline__ long long steps_before(const PagedArgs &a, const SeqTokens &t, int i)
{
    return KV_H * (units_before(a, t, i) + (long long)a.lead * i);
}

__device__ __forceinline__ long long range_begin(const PagedStart &s, int c)
{
    return s.quot * c + s.rem * c / PG_RANGES;
}

// The start of range c, by all THREADS threads of the CTA: per-thread sums over
// a stretch of sequences, a block scan, then the owner of the range's first unit
// walks its stretch. `scan` is shared scratch of THREADS / 32 + 1 values.
template <int THREADS>
__device__ __forceinline__ void find_start(const PagedArgs &a, int c, long long *scan, PagedStart *out)
{
    const PagedBatch &b = a.b;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (b.B + THREADS - 1) / THREADS, s0 = min(tid * per, b.B), s1 = min(s0 + per, b.B);
    long long mine = 0;
    for (int s = s0; s < s1; ++s) {
        const SeqTokens t = seq_tokens(b, s);
        mine += steps_before(a, t, seq_tiles(a, t));
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        long long v = lane < THREADS / 32 ? scan[lane] : 0;
#pragma unroll
        for (int o = 1; o < THREADS / 32; o <<= 1) {
            const long long w = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += w;
        }
        if (lane < THREADS / 32) scan[lane] = v;
    }
    __syncthreads();
    const long long total = scan[THREADS / 32 - 1], before = incl - mine + (warp > 0 ? scan[warp - 1] : 0);
    PagedStart cuts;
    if (total < 0x7FFFFFFF) {                      // a 64-bit division takes four times as long
        cuts.quot = (uint32_t)total / PG_RANGES;
        cuts.rem = (int)((uint32_t)total % PG_RANGES);
    } else {
        cuts.quot = total / PG_RANGES;
        cuts.rem = (int)(total % PG_RANGES);
    }
    const long long u = range_begin(cuts, c);
    if (tid == 0) {
        out->quot = cuts.quot;
        out->rem = cuts.rem;
        out->seq = out->tile = out->head = out->step = 0;
    }
    __syncthreads();
    if (mine > 0 && u >= before && u < before + mine) {
        long long left = u - before;
        int s = s0;
        SeqTokens t = seq_tokens(b, s);
        for (;;) {
            const long long n = steps_before(a, t, seq_tiles(a, t));
            if (left < n) break;
            left -= n;
            t = seq_tokens(b, ++s);
        }
        int lo = 0, hi = seq_tiles(a, t) - 1;         // the tile: largest i with steps_before(i) <= left
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (steps_before(a, t, mid) <= left) lo = mid;
            else hi = mid - 1;
        }
        left -= steps_before(a, t, lo);
        const int n = tile_units(a, t, lo) + a.lead;
        out->seq = s;
        out->tile = lo;
        out->head = (int)(left / n);
        out->step = (int)(left % n);
        out->t = t;
    }
    __syncthreads();
}

// Walks a range piece by piece: units [unit, unit + len) of item (seq, tile, head).
// A walk that has found no (further) piece has len = 0.
struct PieceWalk {
    int seq, tile, head, unit, len, units;        // units of the whole item
    long long left;                               // steps of the range after this piece
    SeqTokens t;
    bool first;                                   // the range's first piece

    // The piece from step `from` of the current item; empty if only leading steps are left of the range.
    __device__ __forceinline__ void cut(const PagedArgs &a, int from, long long avail)
    {
        units = tile_units(a, t, tile);
        const int to = (int)min((long long)(units + a.lead), from + avail);
        left = avail - (to - from);
        unit = max(from - a.lead, 0);
        len = max(to - a.lead, 0) - unit;
    }
    __device__ __forceinline__ void begin(const PagedArgs &a, const PagedStart &s, long long count)
    {
        seq = s.seq;
        tile = s.tile;
        head = s.head;
        first = true;
        t = s.t;
        cut(a, s.step, count);                    // ends inside the leading steps: no piece, and left = 0
    }
    // Whether the range has a piece after this one: what is left reaches past the
    // next item's leading steps.
    __device__ __forceinline__ bool more(const PagedArgs &a) const { return left > a.lead; }
    // Moves to the next piece; only if there is one.
    __device__ __forceinline__ void next(const PagedArgs &a)
    {
        first = false;
        if (++head == KV_H) {
            head = 0;
            if (++tile >= seq_tiles(a, t)) {
                tile = 0;
                do {
                    if (seq + 1 >= a.b.B) {        // not while steps are left, unless the lengths changed during the call
                        len = 0;
                        left = 0;
                        return;
                    }
                    t = seq_tokens(a.b, ++seq);
                } while (t.n == 0);
            }
        }
        cut(a, 0, left);
    }
    __device__ __forceinline__ bool whole() const { return unit == 0 && len == units; }
    __device__ __forceinline__ int tokens(const PagedArgs &a) const { return min(a.tok, t.n - (tile << a.tok_log2)); }
};

// A walk over the units of a range, one at a time.
struct UnitWalk {
    PieceWalk w;
    int j;
    __device__ __forceinline__ void begin(const PagedArgs &a, const PagedStart &s, long long count)
    {
        w.begin(a, s, count);
        j = 0;
    }
    __device__ __forceinline__ bool last(const PagedArgs &a) const { return j + 1 >= w.len && !w.more(a); }
    __device__ __forceinline__ void next(const PagedArgs &a)
    {
        if (++j == w.len) {
            w.next(a);
            j = 0;
        }
    }
};

// ---- small device helpers of the paged kernels

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Pairs of fp32 in one instruction, each rounded as its scalar form.
__device__ __forceinline__ uint64_t pair2(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpair2(uint64_t r)
{
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(r));
    return v;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3, %4}], [%5];"
                 ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}

__device__ __forceinline__ void store8_out(float *p, const float (&x)[8])
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8_out(bf16 *p, const float (&x)[8])
{
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                                               pack_bf16(x[6], x[7]));
}
// A load of global memory that the kernel before may have written (not through the read-only path), free to move
// past stores to shared memory.
__device__ __forceinline__ uint4 load_global(const uint4 *p)
{
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
// inv * sigmoid(g) in four instructions, two of them special functions (a few 2^-23
// relative). Epilogues wait for these: with expf and a division in full an item's
// 32,768 outputs took three times as long, with a Newton reciprocal twice.
__device__ __forceinline__ float gate1(float g, float inv)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(1.0f + ex2(-1.4426950408889634f * g)));
    return y * inv;
}
__device__ __forceinline__ void gate8(const uint4 u, float (&o)[8], float inv)
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] *= gate1(__uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16)), inv);
}
// Normalised output times the gate (if there is one), 4 dims from dim d of (packed row m, head h).
template <typename TO>
__device__ __forceinline__ void finish4(const PagedArgs &a, uint2 gate, int m, int h, int d, float4 o, float inv)
{
    float s[4] = {inv, inv, inv, inv};
    if (a.gate != nullptr) {
        s[0] = gate1(__uint_as_float(gate.x << 16), inv);
        s[1] = gate1(__uint_as_float(gate.x & 0xFFFF0000u), inv);
        s[2] = gate1(__uint_as_float(gate.y << 16), inv);
        s[3] = gate1(__uint_as_float(gate.y & 0xFFFF0000u), inv);
    }
    store4(static_cast<TO *>(a.out) + ((size_t)m * KV_HQ + h) * KV_D + d,
           make_float4(o.x * s[0], o.y * s[1], o.z * s[2], o.w * s[3]));
}

// ---- host side, gdn_paged.cu and gdn_paged_q4.cu

bool encode_tiled(CUtensorMap *map, CUtensorMapDataType dt, int rank, const void *base, const cuuint64_t *dims,
                  const cuuint64_t *strides, const cuuint32_t *box, CUtensorMapSwizzle swizzle);
cudaError_t launch_paged_q4(const PagedArgs &a, gdn_dtype out_dt, cudaStream_t s);

// The kernel's shared-memory attribute, set once per device.
template <auto KERNEL> static cudaError_t smem_attr_once(size_t bytes)
{
    static std::mutex mu;
    static bool done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 0 || dev >= 64 || !done[dev]) {
        e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
    }
    return e;
}

}  // namespace gdn
