// gdn_kv.cuh -- the paged key/value cache of the full-attention layers, as the
// kernels that write it (gdn_kv.cu) and read it (gdn_paged.cu) see it: the
// formats' addresses and the map from packed tokens to cache rows.
#pragma once

#include "gdn_common.cuh"

namespace gdn {

constexpr int KV_HQ = GDN_ATTN_Q_HEADS;           // 16 query heads
constexpr int KV_H = GDN_ATTN_KV_HEADS;           // 2 KV heads
constexpr int KV_D = GDN_ATTN_HEAD_DIM;           // 256
constexpr int KV_G = KV_HQ / KV_H;                // 8 query heads per KV head
constexpr int REC_ROWS = GDN_KV_RECORD_ROWS;      // 16 rows per 4-bit record
constexpr uint32_t REC_BYTES = GDN_KV_RECORD_BYTES;
constexpr uint32_t REC_V = REC_ROWS * 128;        // value codes of a record
constexpr uint32_t REC_KSZ = 2 * REC_ROWS * 128;  // key (s, z) pairs, 16 bytes per row
constexpr uint32_t REC_VSZ = REC_KSZ + REC_ROWS * 16;
static_assert(REC_VSZ + REC_ROWS * 16 == REC_BYTES, "4-bit record layout");

struct PagedBatch {
    const int32_t *table, *ctx, *cu;
    int B, M, max_q, max_pages, num_pages, page, page_log2;
};

inline PagedBatch paged_batch(const gdn_paged_batch &b, const gdn_kv_cache &c)
{
    int lg = 0;
    while ((1 << lg) < c.page_size) ++lg;
    return PagedBatch{b.page_table, b.ctx_len, b.cu_q, b.B, b.M, b.max_q, b.max_pages, c.num_pages, c.page_size, lg};
}

// Sequence of packed row m and its position in that sequence's context, or seq
// = -1 for padding rows. Called by whole warps with the same m: with cu_q the
// number of entries cu[1..B] at or below m is found by probing 32 of them at a
// time (one round up to 32 sequences, two up to 1024).
struct TokenPlace {
    int seq, pos;
};
__device__ __forceinline__ TokenPlace token_place(const PagedBatch &b, int m, int lane)
{
    if (b.cu == nullptr) return m < b.B ? TokenPlace{m, __ldg(b.ctx + m) - 1} : TokenPlace{-1, 0};
    int lo = 0, hi = b.B;                          // the count lies in [lo, hi]
    while (lo < hi) {
        const int step = (hi - lo + 31) >> 5;
        const int i = lo + (lane + 1) * step;      // probes cu[i]
        const bool below = i <= hi && __ldg(b.cu + i) <= m;
        const int k = __popc(__ballot_sync(0xffffffffu, below));
        lo += k * step;
        hi = min(hi, lo + step - 1);
    }
    if (lo >= b.B) return TokenPlace{-1, 0};
    return TokenPlace{lo, __ldg(b.ctx + lo) - (__ldg(b.cu + lo + 1) - m)};
}

// Row of the cache that holds position `pos` of sequence `seq`, as page and row
// within the page; page = -1 where there is none.
__device__ __forceinline__ int cache_page(const PagedBatch &b, int seq, int pos)
{
    if (pos < 0 || (pos >> b.page_log2) >= b.max_pages) return -1;
    const int p = __ldg(b.table + (size_t)seq * b.max_pages + (pos >> b.page_log2));
    return (unsigned)p < (unsigned)b.num_pages ? p : -1;
}

// Element offset of row `off` of (page, head) in a bf16 cache.
__device__ __forceinline__ size_t row_bf16(const PagedBatch &b, int page, int head, int off)
{
    return ((((size_t)page * KV_H + head) << b.page_log2) + off) * KV_D;
}
// Byte offset of the record of row `off` of (page, head) in a 4-bit cache.
__device__ __forceinline__ size_t record_of(const PagedBatch &b, int page, int head, int off)
{
    return (((((size_t)page * KV_H + head) << b.page_log2) + off) / REC_ROWS) * REC_BYTES;
}

}  // namespace gdn
