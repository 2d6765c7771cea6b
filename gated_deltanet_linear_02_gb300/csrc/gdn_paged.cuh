// gdn_paged.cuh -- how the paged attention kernels share out their work.
//
// An item is 16 consecutive new tokens of one sequence (the last one may have
// fewer) and one KV head: up to 128 query rows (8 heads x 16 tokens) that read
// the same keys and values. Its units are the 128-position tiles of the context
// that its last token sees, at least one. The units of all items, in order of
// sequence, tokens, head and position, are cut into one even range per CTA,
// wherever that falls: contexts of any mix of lengths and batches of any size
// keep every SM busy to the end. An item inside one CTA's range is finished
// there; the pieces of an item that spans CTAs go to the workspace as
// unnormalised outputs with their maximum and sum, at most two per CTA (its
// first and its last), and a second kernel joins them. Lengths are read on the
// device, so a captured call follows them from replay to replay.
#pragma once

#include "gdn_kv.cuh"

namespace gdn {

constexpr int PG_TOK = 16;                        // tokens per item, at most
constexpr int PG_TILE = 128;                      // positions per unit
constexpr int PG_ROWS = PG_TOK * KV_G;            // 128 query rows
constexpr int PG_MAX_CTAS = 304;                  // ranges, at most (two per SM of 152)

struct PagedArgs {
    PagedBatch b;
    const void *ck, *cv;
    const bf16 *q, *gate;
    long long gate_row, gate_head;
    void *out;
    struct PagedStart *start;                     // [ranges]
    float *part_o;                                // [2 * ranges][rows][256]
    float *part_ml;                               // [2 * ranges][rows][2]
    int rows;                                     // rows per piece in the workspace: 8 min(max_q, 16)
    int ranges;
    int lead;                                     // leading steps of an item
};

// Where a range starts; `total` is the number of steps of the whole call.
struct PagedStart {
    long long total;
    int seq, tile, head, step;
};

// One sequence's new tokens: packed rows [row0, row0 + n) at positions first,
// first + 1, ...
struct SeqTokens {
    int row0, n, first;
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
__device__ __forceinline__ int tile_sees(const PagedBatch &b, const SeqTokens &t, int i)
{
    return min(t.first + min(PG_TOK * (i + 1), t.n), b.max_pages << b.page_log2);
}
__device__ __forceinline__ int tile_units(const PagedBatch &b, const SeqTokens &t, int i)
{
    return max((tile_sees(b, t, i) + PG_TILE - 1) / PG_TILE, 1);
}

// Units of tiles 0 .. i-1, per head. With x = floor((first + 127) / 16), whole
// tile j (from 1) has floor((x + j) / 8) units, and the sum of floor(m / 8) over
// m = 0 .. 8 q + r is 4 q (q - 1) + q (r + 1). Contexts that start below 0 or
// end past the table are summed term by term.
__device__ __forceinline__ long long units_before(const PagedBatch &b, const SeqTokens &t, int i)
{
    if (t.first < 0 || t.first + t.n > (b.max_pages << b.page_log2)) {
        long long u = 0;
        for (int j = 0; j < i; ++j) u += tile_units(b, t, j);
        return u;
    }
    const int tiles = (t.n + PG_TOK - 1) / PG_TOK, whole = min(i, t.n / PG_TOK);
    auto sum = [](long long m) { const long long q = m >> 3; return 4 * q * (q - 1) + q * ((m & 7) + 1); };
    const int x = (t.first + PG_TILE - 1) / PG_TOK;
    long long u = sum(x + whole) - sum(x);
    if (i == tiles && whole < tiles) u += tile_units(b, t, tiles - 1);
    return u;
}
__device__ __forceinline__ int seq_tiles(const SeqTokens &t) { return (t.n + PG_TOK - 1) / PG_TOK; }
// Steps of tiles 0 .. i-1, both heads.
__device__ __forceinline__ long long steps_before(const PagedArgs &a, const SeqTokens &t, int i)
{
    return KV_H * (units_before(a.b, t, i) + (long long)a.lead * i);
}

__device__ __forceinline__ long long range_begin(long long total, int c, int ranges)
{
    return total / ranges * c + total % ranges * c / ranges;
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
        mine += steps_before(a, t, seq_tiles(t));
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
    const long long u = range_begin(total, c, a.ranges);
    if (tid == 0) {
        out->total = total;
        out->seq = out->tile = out->head = out->step = 0;
    }
    __syncthreads();
    if (mine > 0 && u >= before && u < before + mine) {
        long long left = u - before;
        int s = s0;
        SeqTokens t = seq_tokens(b, s);
        for (;;) {
            const long long n = steps_before(a, t, seq_tiles(t));
            if (left < n) break;
            left -= n;
            t = seq_tokens(b, ++s);
        }
        int lo = 0, hi = seq_tiles(t) - 1;         // the tile: largest i with steps_before(i) <= left
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (steps_before(a, t, mid) <= left) lo = mid;
            else hi = mid - 1;
        }
        left -= steps_before(a, t, lo);
        const int n = tile_units(b, t, lo) + a.lead;
        out->seq = s;
        out->tile = lo;
        out->head = (int)(left / n);
        out->step = (int)(left % n);
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
        units = tile_units(a.b, t, tile);
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
        t = seq_tokens(a.b, seq);
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
            if (++tile >= seq_tiles(t)) {
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
    __device__ __forceinline__ int tokens() const { return min(PG_TOK, t.n - PG_TOK * tile); }
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

}  // namespace gdn
