// gdn_paged.cu -- causal attention of new tokens over the paged cache, steps 5-6
// of section "Full-attention block" of "qwen35moe -- Forward-Pass Design
// (Pantheon port)", on 5th-generation tensor cores. gdn_paged.cuh describes how
// the work is shared out: pieces of up to 128 query rows (16 tokens x the 8
// heads of a KV head) over 128-position tiles of the context.
//
// Per unit (one tile), with M = 128 query rows:
//   S = Q K^T (N = 128 positions, K = 256 dims), fp32 in tensor memory;
//   P = 2^((S - m) log2 e / 16), rounded to bf16, over S's own columns;
//   O += P V (N = 256 dims, K = 128 positions), fp32 in tensor memory,
// m the row's reference maximum and l its sum of P. O is rescaled only when a
// row's maximum passes m by more than 8 (in powers of two): P then stays below
// 2^8, l and O lose nothing in fp32, and the rescale, a round trip of the whole
// accumulator, happens a few times per context instead of at every tile.
//
// Roles in a CTA (one per SM, 384 threads, 640 with 4-bit pages):
//  - warp 0, TMA producer: 32 KiB stages of 128 positions x 128 dims (keys low,
//    high, values low, high), one box per page and 64 dims, in a ring of four;
//    the next tile's keys ahead of this tile's values, as the MMAs use them;
//  - warps 1 and 2, one lane each, issue the two products: each waits for its own
//    operands while the other's instructions run (one issuer for both left the
//    tensor core idle for half of every unit: 2.6 us instead of 1.6);
//  - warps 4-11, two threads per query row, each with half of a tile's positions
//    and half of the output's dims: softmax, rescale, and the epilogue (normalise
//    and gate, or store the piece's unnormalised output);
//  - warps 12-19, with 4-bit pages only: codes to bf16. The producer then copies
//    the eight records' key or value codes of a tile (18 KiB, a quarter of the
//    values) into one of two buffers, and these warps write the stages, a ring of
//    three. With four warps 173 us where eight take 162, for three sequences
//    of up to 517 tokens over contexts of up to 6,001.
// Values that are not finite: a weight of 0 times infinity or NaN is NaN, so a value
// row may only enter the product as it is if all 16 tokens of the item see it. Rows
// that none sees become zeros, and of those that some see (the item's own tokens, at
// most 15) the infinities and NaN do; the epilogue then adds them to the rows that
// see them. Looking at these rows is a few instructions per item.
// Tensor memory: two S buffers (P over their first half) and O, all 512 columns.
//
// Bound: for one token per sequence by HBM (1 KiB of keys and values per position
// and KV head; the 120 unused rows cost tensor time that hides behind it): 256
// contexts of up to 4,096 take 245 us, 6.6 TB/s. For prompts by the shared-memory
// port, which carries Q, K, V and the TMA writes of a tile in about 2,500 cycles
// against 2,048 of tensor work: 1.59 us per tile over contexts of 16,384 (1,600
// TFLOP/s), and about 9 us per item for its epilogue, its tile on the diagonal and
// the start of the next, during which the products wait: a prompt of 4,096 tokens
// takes 137 us. With 4-bit pages the port also carries the codes, and the logic
// pipe their expansion: 2.7 us per tile.
#include <cuda.h>

#include "gdn_async.cuh"
#include "gdn_paged.cuh"
#include "gdn_tc.cuh"

namespace gdn {

__device__ unsigned int g_paged_error;            // GDN_ERR_TIMEOUT if a bounded wait gave up

constexpr int FA_DEQUANT = 256;                   // threads that turn codes to bf16
constexpr int fa_threads(bool q4) { return 384 + (q4 ? FA_DEQUANT : 0); }
constexpr uint32_t FA_BOX = PG_TILE * 128;        // 128 rows x 64 dims of bf16: 16 KiB
constexpr uint32_t FA_STAGE_BYTES = 2 * FA_BOX;   // 128 dims: 32 KiB
constexpr uint32_t FA_S = 0, FA_O = 256;          // tensor memory columns: S buffers at 0 and 128, O at 256

// Shared memory. 4-bit pages take one stage less and half of the epilogue's boxes
// for two tiles of codes as they are stored: eight records' key or value parts.
constexpr uint32_t FA_CODES = 2048, FA_TILE_BYTES = 8 * (2048 + 256);
template <bool Q4> struct Fa {
    static constexpr int STAGES = Q4 ? 3 : 4;
    static constexpr int PART = Q4 ? 32 : 64;     // dims that an epilogue box holds
    static constexpr uint32_t BOX = 32 * PART * 2;   // per softmax warp
    static constexpr uint32_t Q = 0;              // Q: 4 boxes of 64 dims
    static constexpr uint32_t RING = 4 * FA_BOX;
    static constexpr uint32_t EPI = RING + STAGES * FA_STAGE_BYTES;
    static constexpr uint32_t TILES = EPI + 8 * BOX;
    static constexpr uint32_t SMALL = TILES + (Q4 ? 2 * FA_TILE_BYTES : 0);
};

struct FaSmall {
    uint64_t full[4], empty[4];
    uint64_t q_full, q_empty, s_full[2], p_full[2], pv_done[2], o_empty, done[2];
    uint64_t t_full[2], t_empty[2];               // tiles of codes
    int t_sees[2];                                // positions of the tile that the item sees, and << 8 of those that
                                                  // all its tokens see (keys: the same); below 0: no more tiles
    long long scan[fa_threads(true) / 32 + 1];
    uint32_t top[2][2][128];                      // by unit parity and group: a row's maximum
    PagedStart start;
    uint32_t tmem;
    int abort;
    int poison;                                   // values that are not finite have been set to zero
};
// Slack to align the block to 1 KiB. Dynamic shared memory starts on such a boundary
// as it is; the kernel checks that the slack is enough.
constexpr uint32_t FA_SLACK = 512;
template <bool Q4> constexpr size_t FA_SMEM = Fa<Q4>::SMALL + sizeof(FaSmall) + FA_SLACK;
static_assert(FA_SMEM<false> <= 232448 && FA_SMEM<true> <= 232448, "shared memory of one CTA");

// Two bf16 values of a word's codes t and t + 4: s c + z with one rounding (128 + c
// by one logic operation, minus 128 exactly).
__device__ __forceinline__ uint32_t value_pair(uint32_t w, int t, uint32_t s2, uint32_t z2)
{
    uint32_t c, v;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(c) : "r"(w >> (4 * t)), "r"(0x000F000Fu), "r"(0x43004300u));   // (w & b) | c
    asm("sub.rn.bf16x2 %0, %0, %1;" : "+r"(c) : "r"(0x43004300u));
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(v) : "r"(c), "r"(s2), "r"(z2));
    return v;
}

// Marks (bits 15 and 31) of the two bf16 of a word that are infinite or NaN.
__device__ __forceinline__ uint32_t not_finite(uint32_t w) { return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u; }

// Which of the 16 values from dim d of position p's value row are +infinity (bits 0-15) or -infinity (16-31); both:
// NaN. Plain loads: the append before this kernel may write the row while this one has started.
template <bool Q4> __device__ __forceinline__ uint32_t poison_of(const PagedArgs &a, int seq, int head, int p, int d)
{
    const int page = cache_page(a.b, seq, p), off = p & (a.b.page - 1);
    if (page < 0) return 0u;
    if (Q4) {
        const unsigned char *rec = static_cast<const unsigned char *>(a.ck) + record_of(a.b, page, head, off);
        const uint32_t sz = *(reinterpret_cast<const uint32_t *>(rec + REC_VSZ + (off % REC_ROWS) * 16) + d / 64);
        return not_finite(sz) != 0u ? 0xFFFFFFFFu : 0u;
    }
    const uint16_t *row = static_cast<const uint16_t *>(a.cv) + row_bf16(a.b, page, head, off) + d;
    uint32_t m = 0u;
#pragma unroll 1
    for (int k = 0; k < 16; ++k) {
        const uint32_t x = row[k];
        if ((x & 0x7F80u) == 0x7F80u) m |= (x & 0x7Fu) != 0u ? 0x10001u << k : 1u << (k + 16 * (x >> 15));
    }
    return m;
}

// Brings a tensor map near before its first use.
__device__ __forceinline__ void prefetch_map(const CUtensorMap *m) { asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory"); }

template <int N> __device__ __forceinline__ void set_registers_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void set_registers_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

template <typename TO, bool Q4>
__global__ void __launch_bounds__(fa_threads(Q4), 1) attn_paged_kernel(const __grid_constant__ CUtensorMap qmap,
                                                                   const __grid_constant__ CUtensorMap kmap,
                                                                   const __grid_constant__ CUtensorMap vmap,
                                                                   const PagedArgs a)
{
    extern __shared__ unsigned char smem_raw[];
    const uint32_t shift = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
    if (shift > FA_SLACK) {
        if (threadIdx.x == 0) atomicExch(&g_paged_error, (unsigned int)GDN_ERR_TIMEOUT);
        return;
    }
    unsigned char *blk = smem_raw + shift;
    FaSmall &ss = *reinterpret_cast<FaSmall *>(blk + Fa<Q4>::SMALL);
    const uint32_t sb = smem_u32(blk);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const PagedBatch &b = a.b;
    const int cap = b.max_pages << b.page_log2;

    if (tid == 0) {
        for (int s = 0; s < Fa<Q4>::STAGES; ++s) {
            mbar_init(smem_u32(&ss.full[s]), Q4 ? FA_DEQUANT : 1);
            mbar_init(smem_u32(&ss.empty[s]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&ss.s_full[i]), 1);
            mbar_init(smem_u32(&ss.p_full[i]), 256);
            mbar_init(smem_u32(&ss.pv_done[i]), 1);
            mbar_init(smem_u32(&ss.done[i]), 1);
            mbar_init(smem_u32(&ss.t_full[i]), 32);
            mbar_init(smem_u32(&ss.t_empty[i]), FA_DEQUANT);
        }
        mbar_init(smem_u32(&ss.q_full), 1);
        mbar_init(smem_u32(&ss.q_empty), 1);
        mbar_init(smem_u32(&ss.o_empty), 256);
        ss.abort = ss.poison = 0;
        fence_mbar_init();
    }
    if (!Q4 && tid == 32) {                        // 1% of a prompt; none with 4-bit pages, whose first copies are of codes
        prefetch_map(&qmap);
        prefetch_map(&kmap);
        prefetch_map(&vmap);
    }
    if (warp == 3) {
        tc::tmem_alloc(smem_u32(&ss.tmem), 512);
        tc::tmem_relinquish();
    }
    grid_dep_wait();
    grid_dep_launch();
    find_start<fa_threads(Q4)>(a, blockIdx.x, ss.scan, &ss.start);   // ends in a CTA barrier
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = ss.tmem;
    const PagedStart st = ss.start;
    if (tid == 0) a.start[blockIdx.x] = st;
    const long long count = range_begin(st, blockIdx.x + 1) - range_begin(st, blockIdx.x);
    const volatile int &aborted = ss.abort;
    auto stage = [&](uint32_t i) { return sb + Fa<Q4>::RING + (i % Fa<Q4>::STAGES) * FA_STAGE_BYTES; };
    auto wait_full = [&](uint32_t i) {
        return mbar_wait_sleep(smem_u32(&ss.full[i % Fa<Q4>::STAGES]), (i / Fa<Q4>::STAGES) & 1);
    };

    PieceWalk first;
    if (count > 0) first.begin(a, st, count);
    if (count > 0 && first.len > 0) {
        // registers with 4-bit pages: 64 + 2 x 152 + 2 x 56 of the 5 x 96 launched with
        if (warp < 4) {
            if (Q4) set_registers_down<64>();
            if (warp == 0) {
                // ---- TMA producer. Stage order: K(0), then K(u + 1), V(u) for each u.
                UnitWalk kw;
                kw.begin(a, st, count);
                const int seg = lane >> 1, box = lane & 1, nseg = PG_TILE >> b.page_log2;
                const uint32_t seg_dst = (uint32_t)seg * ((uint32_t)b.page * 128) + box * FA_BOX;
                uint32_t i = 0, piece = 0;
                bool ok = true;
                // row of the cache tensors where this lane's segment of the unit starts; segments past
                // what the item sees are not loaded, bad page ids load past the end (zeros)
                auto segment = [&](int &row, int &loaded) {
                    const int p = (kw.w.unit + kw.j) * PG_TILE;
                    const int sees = tile_sees(a, kw.w.t, kw.w.tile);
                    loaded = min(nseg, max(0, (sees - p + b.page - 1) >> b.page_log2));
                    row = 0;
                    if (seg < loaded) {
                        const int page = cache_page(b, kw.w.seq, p + seg * b.page);
                        row = page < 0 ? (b.num_pages * KV_H) << b.page_log2 : ((page * KV_H + kw.w.head) << b.page_log2);
                    }
                };
                auto load = [&](const CUtensorMap *m, int row, int loaded) {
                    for (int half = 0; half < 2 && ok; ++half, ++i) {
                        if (i >= Fa<Q4>::STAGES)
                            ok = mbar_wait_sleep(smem_u32(&ss.empty[i % Fa<Q4>::STAGES]), (i / Fa<Q4>::STAGES - 1) & 1);
                        ok = __all_sync(0xffffffffu, ok && !aborted);
                        if (!ok) break;
                        const uint32_t bar = smem_u32(&ss.full[i % Fa<Q4>::STAGES]);
                        if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)loaded * b.page * 256);
                        __syncwarp();
                        if (seg < loaded) tma_load_2d(stage(i) + seg_dst, m, half * 128 + box * 64, row, bar);
                    }
                };
                auto load_q = [&](int row0, int head) {
                    if (piece > 0) ok = mbar_wait_sleep(smem_u32(&ss.q_empty), (piece - 1) & 1);
                    ok = __all_sync(0xffffffffu, ok && !aborted);
                    if (ok && lane == 0) {
                        const uint32_t bar = smem_u32(&ss.q_full);
                        mbar_arrive_expect_tx(bar, 4 * FA_BOX);
                        for (int c = 0; c < 4; ++c)
                            tma_load_3d(sb + Fa<Q4>::Q + c * FA_BOX, &qmap, 64 * c, KV_G * head, row0, bar);
                    }
                    ++piece;
                };
                if (!Q4) {
                    load_q(kw.w.t.row0 + PG_TOK * kw.w.tile, kw.w.head);
                    int row, loaded;
                    segment(row, loaded);
                    if (ok) load(&kmap, row, loaded);
                    while (ok) {
                        const int vrow = row, vloaded = loaded;
                        const bool more = !kw.last(a);
                        if (more) {
                            kw.next(a);
                            segment(row, loaded);
                            if (kw.j == 0) load_q(kw.w.t.row0 + PG_TOK * kw.w.tile, kw.w.head);
                            if (ok) load(&kmap, row, loaded);
                        }
                        if (ok) load(&vmap, vrow, vloaded);
                        if (!more) break;
                    }
                } else {
                    // tiles of codes in the same order: the keys of the next unit, unless those of two are
                    // ahead of their values (q0, q1), else the values of the oldest. Lane k: record k.
                    struct Unit {
                        int rec, sees, all, row0, head;   // the lane's record (-1: zeros, -2: none), positions seen (by all), the queries
                        bool first;
                    };
                    Unit q0 = {}, q1 = {}, tile;
                    int ahead = 0, entry = 0;
                    bool have = true;
                    auto look_up = [&]() {             // page table entry of the lane's record of the unit kw is at
                        const int p = (kw.w.unit + kw.j) * PG_TILE + 16 * lane;
                        if (lane < 8 && p < tile_sees(a, kw.w.t, kw.w.tile))
                            entry = __ldg(b.table + (size_t)kw.w.seq * b.max_pages + (p >> b.page_log2));
                    };
                    look_up();
                    for (uint32_t n = 0;; ++n) {
                        const bool value = !(ahead < 2 && have);
                        if (!value) {
                            const int p = (kw.w.unit + kw.j) * PG_TILE, at = (kw.w.head << b.page_log2) + ((p + 16 * lane) & (b.page - 1));
                            tile.sees = max(min(tile_sees(a, kw.w.t, kw.w.tile) - p, PG_TILE), 0);
                            tile.rec = lane >= 8 || 16 * lane >= tile.sees ? -2
                                       : (unsigned)entry < (unsigned)b.num_pages ? (((entry * KV_H) << b.page_log2) + at) >> 4 : -1;
                            tile.all = min(max(kw.w.t.first + PG_TOK * kw.w.tile + 1 - p, 0), tile.sees);
                            tile.row0 = kw.w.t.row0 + PG_TOK * kw.w.tile;
                            tile.head = kw.w.head;
                            tile.first = kw.j == 0;
                            (ahead++ == 0 ? q0 : q1) = tile;
                            have = !kw.last(a);
                            if (have) {
                                kw.next(a);
                                look_up();
                            }
                            if (tile.first) load_q(tile.row0, tile.head);
                        } else if (ahead > 0) {
                            tile = q0;
                            q0 = q1;
                            --ahead;
                        } else {
                            tile.sees = -1;            // no more
                            tile.rec = -2;
                        }
                        if (n >= 2) ok = ok && mbar_wait_sleep(smem_u32(&ss.t_empty[n & 1]), ((n >> 1) - 1) & 1);
                        ok = __all_sync(0xffffffffu, ok && !aborted);
                        if (!ok) break;
                        const uint32_t bar = smem_u32(&ss.t_full[n & 1]);
                        const uint32_t at = Fa<Q4>::TILES + (n & 1) * FA_TILE_BYTES;
                        if (lane == 0) ss.t_sees[n & 1] = tile.sees < 0 ? -1 : tile.sees | (value ? tile.all : tile.sees) << 8;
                        if (tile.rec >= 0) {
                            const unsigned char *src = static_cast<const unsigned char *>(a.ck) + (size_t)tile.rec * REC_BYTES;
                            mbar_arrive_expect_tx(bar, FA_CODES + 256);
                            bulk_g2s(sb + at + lane * FA_CODES, src + (value ? REC_V : 0u), FA_CODES, bar);
                            bulk_g2s(sb + at + 8 * FA_CODES + lane * 256, src + (value ? REC_VSZ : REC_KSZ), 256, bar);
                        } else {
                            if (tile.rec == -1) {      // a page id outside the cache: zeros
                                const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
                                for (uint32_t k = 0; k < FA_CODES; k += 16) *reinterpret_cast<uint4 *>(blk + at + lane * FA_CODES + k) = zero;
                                for (uint32_t k = 0; k < 256; k += 16) *reinterpret_cast<uint4 *>(blk + at + 8 * FA_CODES + lane * 256 + k) = zero;
                                fence_proxy_async_smem();
                            }
                            mbar_arrive(bar);
                        }
                        if (tile.sees < 0) break;
                        i = n + 1;                     // tiles loaded
                    }
                }
                if (!ok) {                             // copies in flight land before the CTA exits
                    if (lane == 0) ss.abort = 1;
                    if (Q4)
                        for (uint32_t k = i > 2 ? i - 2 : 0; k < i; ++k) mbar_wait_sleep(smem_u32(&ss.t_full[k & 1]), (k >> 1) & 1);
                    else
                        for (uint32_t k = i > Fa<Q4>::STAGES ? i - Fa<Q4>::STAGES : 0; k < i; ++k) wait_full(k);
                    if (piece > 0) mbar_wait_sleep(smem_u32(&ss.q_full), (piece - 1) & 1);
                }
            } else if (warp == 1) {
                // ---- issuer of S(u) = Q K^T
                if (lane == 0) {
                    const uint32_t id = tc::instr_desc(tc::FMT_BF16, 128, PG_TILE);
                    UnitWalk w;
                    w.begin(a, st, count);
                    uint32_t i = 0, piece = 0;
                    bool ok = true;
                    for (uint32_t u = 0; ok; ++u) {
                        if (w.j == 0) ok = mbar_wait_sleep(smem_u32(&ss.q_full), piece++ & 1);
                        // the buffer holds P of unit u - 2 until its product is complete
                        if (u >= 2) ok = ok && mbar_wait_sleep(smem_u32(&ss.pv_done[u & 1]), ((u - 2) >> 1) & 1);
                        if (u == 1) i = 2;
                        for (int half = 0; half < 2 && ok; ++half, ++i) {
                            ok = wait_full(i) && !aborted;
                            if (!ok) break;
                            tc::fence_after_sync();
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk)
                                tc::mma_f16(tm + FA_S + (u & 1) * 128,
                                            tc::sw128_desc(sb + Fa<Q4>::Q + (2 * half + (kk >> 2)) * FA_BOX + (kk & 3) * 32),
                                            tc::sw128_desc(stage(i) + (kk >> 2) * FA_BOX + (kk & 3) * 32), id,
                                            half + kk > 0 ? 1u : 0u);
                            tc::mma_commit(smem_u32(&ss.empty[i % Fa<Q4>::STAGES]));
                        }
                        if (!ok) break;
                        tc::mma_commit(smem_u32(&ss.s_full[u & 1]));
                        if (w.j + 1 == w.w.len) tc::mma_commit(smem_u32(&ss.q_empty));
                        if (w.last(a)) break;
                        w.next(a);
                        if (u > 0) i += 2;             // the values of unit u - 1 come between
                    }
                    if (!ok) ss.abort = 1;
                    tc::mma_commit(smem_u32(&ss.done[0]));   // every MMA completes before tensor memory is freed
                    mbar_wait_sleep(smem_u32(&ss.done[0]), 0u);
                }
            } else if (warp == 2) {
                // ---- issuer of O += P(u) V
                if (lane == 0) {
                    const uint32_t id = tc::instr_desc(tc::FMT_BF16, 128, 128) | tc::IDESC_B_MN;
                    UnitWalk w;
                    w.begin(a, st, count);
                    uint32_t piece = 0;
                    bool ok = true;
                    for (uint32_t u = 0; ok; ++u) {
                        const bool last = w.last(a);
                        uint32_t i = last ? 4 * u + 2 : 4 * u + 4;   // the keys of unit u + 1 come before
                        if (w.j == 0) {                // O of the piece before has been read
                            if (piece > 0) ok = mbar_wait_sleep(smem_u32(&ss.o_empty), (piece - 1) & 1);
                            ++piece;
                        }
                        ok = ok && mbar_wait_sleep(smem_u32(&ss.p_full[u & 1]), (u >> 1) & 1);
                        for (int half = 0; half < 2 && ok; ++half, ++i) {
                            ok = wait_full(i) && !aborted;
                            if (!ok) break;
                            tc::fence_after_sync();
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk)
                                tc::mma_f16_tmem_a(tm + FA_O + half * 128, tm + FA_S + (u & 1) * 128 + kk * 8,
                                                   tc::sw128_mn_desc(stage(i) + kk * 2048, FA_BOX), id,
                                                   w.j + kk > 0 ? 1u : 0u);
                            tc::mma_commit(smem_u32(&ss.empty[i % Fa<Q4>::STAGES]));
                        }
                        if (!ok) break;
                        tc::mma_commit(smem_u32(&ss.pv_done[u & 1]));
                        if (last) break;
                        w.next(a);
                    }
                    if (!ok) ss.abort = 1;
                    tc::mma_commit(smem_u32(&ss.done[1]));
                    mbar_wait_sleep(smem_u32(&ss.done[1]), 0u);
                }
            }
        } else if (Q4 && warp >= 12) {
            set_registers_down<56>();
            // ---- tiles of codes to bf16 stages: thread t of a warpgroup has row t / 8 and dims 8 (t % 8) ..
            // of each group of every second record, two groups (a stage) at a time. Values and keys are
            // rounded to bf16 here (one rounding), the type that the MMA takes.
            const int t = tid & 127, odd = (warp >> 2) - 3, rr = t >> 3, ch = t & 7;
            bool ok = true;
            uint32_t i = 0;
            for (uint32_t n = 0;; ++n) {
                ok = __all_sync(0xffffffffu, mbar_wait_sleep(smem_u32(&ss.t_full[n & 1]), (n >> 1) & 1) && !aborted);
                if (!ok) break;
                const int mark = *const_cast<const volatile int *>(&ss.t_sees[n & 1]), sees = mark & 255, all = mark >> 8;
                if (mark < 0) break;
                const unsigned char *codes = blk + Fa<Q4>::TILES + (n & 1) * FA_TILE_BYTES + odd * FA_CODES + 16 * t;
                const unsigned char *steps = blk + Fa<Q4>::TILES + (n & 1) * FA_TILE_BYTES + 8 * FA_CODES + odd * 256 + 16 * rr;
                for (int half = 0; half < 2; ++half, ++i) {
                    if (i >= Fa<Q4>::STAGES)
                        ok = mbar_wait_sleep(smem_u32(&ss.empty[i % Fa<Q4>::STAGES]), (i / Fa<Q4>::STAGES - 1) & 1);
                    ok = __all_sync(0xffffffffu, ok && !aborted);
                    if (!ok) break;
                    unsigned char *dst = blk + (stage(i) - sb) + odd * 2048 + rr * 128 + ((ch ^ (rr & 7)) << 4);
                    uint2 code[4], step[4];        // all of them first: the compiler keeps loads behind stores
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        code[k] = *reinterpret_cast<const uint2 *>(codes + 2 * k * FA_CODES + 8 * half);
                        step[k] = *reinterpret_cast<const uint2 *>(steps + 2 * k * 256 + 8 * half);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint2 w = code[k];
                        uint2 z = step[k];
                        if (32 * k + 16 * odd + rr >= all) {
                            if (32 * k + 16 * odd + rr >= sees) {
                                z = make_uint2(0u, 0u);    // past the context: zeros, whatever is there
                            } else {                       // not finite, see above
                                if ((not_finite(z.x) | not_finite(z.y)) != 0u) ss.poison = 1;
                                if (not_finite(z.x) != 0u) z.x = 0u;
                                if (not_finite(z.y) != 0u) z.y = 0u;
                            }
                        }
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            const uint32_t c = g == 0 ? w.x : w.y, sz = g == 0 ? z.x : z.y;
                            const uint32_t s2 = __byte_perm(sz, sz, 0x1010), z2 = __byte_perm(sz, sz, 0x3232);
                            const uint32_t v0 = value_pair(c, 0, s2, z2), v1 = value_pair(c, 1, s2, z2);
                            const uint32_t v2 = value_pair(c, 2, s2, z2), v3 = value_pair(c, 3, s2, z2);
                            *reinterpret_cast<uint4 *>(dst + g * FA_BOX + k * 4096) =
                                make_uint4(__byte_perm(v0, v1, 0x5410), __byte_perm(v2, v3, 0x5410), __byte_perm(v0, v1, 0x7632), __byte_perm(v2, v3, 0x7632));
                        }
                    }
                    fence_proxy_async_smem();
                    mbar_arrive(smem_u32(&ss.full[i % Fa<Q4>::STAGES]));
                }
                if (!ok) break;
                mbar_arrive(smem_u32(&ss.t_empty[n & 1]));
            }
            if (!ok && lane == 0) ss.abort = 1;
        } else {
            if (Q4) set_registers_up<152>();
            // ---- softmax and epilogue: threads r of both groups share query row r of the item; group 0
            // has positions 0-63 of a tile and dims 0-127 of the output, group 1 the others
            const int r = tid & 127, q4 = warp & 3, grp = (warp >> 2) - 1;
            const uint32_t lbase = tm + ((uint32_t)(32 * q4) << 16);
            PieceWalk w = first;
            uint32_t u = 0;
            bool ok = true;
            // O += P V of unit v is complete. Two barriers in turn: S of unit u, which this thread has
            // seen, was issued after that of unit u - 2 completed, so each is one phase behind at most.
            auto wait_pv = [&](uint32_t v) { return mbar_wait_sleep(smem_u32(&ss.pv_done[v & 1]), (v >> 1) & 1); };
            // Barriers of the two warps that share rows; the second is the epilogue's, right behind a first one.
            // They have no limit of their own, so a warp that gives up (ok = false; perhaps alone, where one of
            // its waits ran out or it was the first to see the stop) marks its maxima, sets the stop and arrives
            // at both without waiting, see the end. Its partner's next barriers then open, and behind them it
            // finds the mark or the stop and leaves in the same way.
            auto pair_bar = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(1 + q4) : "memory"); };
            auto pair_bar2 = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(5 + q4) : "memory"); };
            for (;;) {
                const int rows = KV_G * w.tokens(a), sees = tile_sees(a, w.t, w.tile);
                // positions this row sees, and those that all rows see; formed at each use, as registers are short
                auto limit_of = [&]() { return min(w.t.first + PG_TOK * w.tile + (r >> 3) + 1, cap); };
                auto all_see = [&]() { return min(w.t.first + PG_TOK * w.tile + 1, sees); };
                const bool live = 32 * q4 < rows;      // the warp has rows of the item
                float m = -INFINITY, l = 0.0f;
                for (int j = 0; j < w.len; ++j, ++u) {
                    const int p0 = (w.unit + j) * PG_TILE, c0 = p0 + 64 * grp;
                    ok = __all_sync(0xffffffffu, mbar_wait_sleep(smem_u32(&ss.s_full[u & 1]), (u >> 1) & 1) && !aborted);
                    tc::fence_after_sync();
                    if (live) {
                        const uint32_t sc = lbase + FA_S + (u & 1) * 128;
                        float x[2][32];
                        if (ok) {
                            tc::tmem_ld32(sc + 64 * grp, x[0]);
                            tc::tmem_ld32(sc + 64 * grp + 32, x[1]);
                            tc::wait_ld();
                        }
                        const int limit = limit_of();
                        if (__any_sync(0xffffffffu, c0 + 64 > limit)) {
#pragma unroll
                            for (int c = 0; c < 2; ++c)
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    if (c0 + 32 * c + i >= limit) x[c][i] = -INFINITY;
                        }
                        float mx[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            mx[c] = fmaxf(x[c >> 1][16 * (c & 1)], x[c >> 1][16 * (c & 1) + 1]);
#pragma unroll
                            for (int i = 2; i < 16; i += 2)
                                mx[c] = fmaxf(mx[c], fmaxf(x[c >> 1][16 * (c & 1) + i], x[c >> 1][16 * (c & 1) + i + 1]));
                        }
                        // the row's maximum over both groups; a stop is passed on as a NaN that no maximum is
                        float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                        ss.top[u & 1][grp][r] = ok ? __float_as_uint(top) : 0xFFFFFFFFu;
                        tc::fence_before_sync();
                        pair_bar();                    // S has been read by both: P may go over it
                        tc::fence_after_sync();
                        const uint32_t other = ss.top[u & 1][grp ^ 1][r];
                        ok = __all_sync(0xffffffffu, ok && other != 0xFFFFFFFFu);
                        if (!ok) break;
                        top = fmaxf(top, __uint_as_float(other));
                        const bool move = (top - m) * SCORE_SCALE > RESCALE_AT;   // also from m = -inf; never for top = -inf
                        if (__any_sync(0xffffffffu, move)) {
                            const float f = !move ? 1.0f : (m == -INFINITY ? 0.0f : ex2((m - top) * SCORE_SCALE));
                            if (j > 0) {
                                ok = __all_sync(0xffffffffu, wait_pv(u - 1));
                                tc::fence_after_sync();
#pragma unroll 1
                                for (int c = 0; c < 4 && ok; ++c) {
                                    float o[32];
                                    tc::tmem_ld32(lbase + FA_O + 128 * grp + 32 * c, o);
                                    tc::wait_ld();
#pragma unroll
                                    for (int i = 0; i < 32; ++i) o[i] *= f;   // infinities and NaN stay, also where f is 0
                                    tc::tmem_st32(lbase + FA_O + 128 * grp + 32 * c, o);
                                }
                                tc::wait_st();
                            }
                            l *= f;
                            m = move ? top : m;
                        }
                        const float off = m == -INFINITY ? 0.0f : m * SCORE_SCALE;
                        uint64_t sum[2] = {0ull, 0ull};
                        const uint64_t scale2 = pair2(SCORE_SCALE, SCORE_SCALE), off2 = pair2(-off, -off);
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            uint32_t pk[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float2 y = unpair2(fma2(pair2(x[c][2 * i], x[c][2 * i + 1]), scale2, off2));
                                const float e0 = ex2(y.x), e1 = ex2(y.y);
                                sum[i & 1] = add2(sum[i & 1], pair2(e0, e1));
                                pk[i] = pack_bf16(e0, e1);
                            }
                            tc::tmem_st16_u32(sc + 32 * grp + 16 * c, pk);
                        }
                        const float2 s2 = unpair2(add2(sum[0], sum[1]));
                        l += s2.x + s2.y;
                        tc::wait_st();
                    }
                    if (!ok) break;
                    if (!Q4 && p0 + PG_TILE > all_see()) {
                        // Value rows that not every token of the item sees, see above: zeros past the context,
                        // whatever the cache (or an earlier tile) left there, and for values that are not
                        // finite. The previous unit's products are waited for first: they free the stages'
                        // earlier use, without which the phase of `full` would be ambiguous.
                        const uint32_t vi = (j + 1 == w.len && !w.more(a) ? 4 * u + 2 : 4 * u + 4) + grp;
                        ok = u == 0 || wait_pv(u - 1);
                        ok = __all_sync(0xffffffffu, ok && wait_full(vi) && !aborted);
                        if (!ok) break;
                        if (p0 + r >= sees) {
                            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                uint4 *row = reinterpret_cast<uint4 *>(blk + (stage(vi) - sb) + k * FA_BOX + r * 128);
#pragma unroll
                                for (int c = 0; c < 8; ++c) row[c] = zero;
                            }
                        }
                        const int own = max(all_see(), p0) + (r >> 3);   // eight threads for each of at most 15 rows
                        if (own < min(sees, p0 + PG_TILE)) {
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                uint4 *at = reinterpret_cast<uint4 *>(blk + (stage(vi) - sb) + k * FA_BOX + (own - p0) * 128) + (r & 7);
                                uint4 v = *at;
                                if ((not_finite(v.x) | not_finite(v.y) | not_finite(v.z) | not_finite(v.w)) != 0u) {
                                    ss.poison = 1;
                                    v.x &= ~((not_finite(v.x) >> 15) * 0xFFFFu);
                                    v.y &= ~((not_finite(v.y) >> 15) * 0xFFFFu);
                                    v.z &= ~((not_finite(v.z) >> 15) * 0xFFFFu);
                                    v.w &= ~((not_finite(v.w) >> 15) * 0xFFFFu);
                                    *at = v;
                                }
                            }
                        }
                        fence_proxy_async_smem();
                    }
                    tc::fence_before_sync();           // P stored, S read
                    mbar_arrive(smem_u32(&ss.p_full[u & 1]));
                }
                if (!ok) break;
                // Epilogue: this group's 128 dims, 64 at a time. A thread's row lies 512 bytes from its
                // neighbour's, so gates come in and outputs leave through 4 KiB of shared memory per warp,
                // in whole 128-byte lines. The gates are read (plainly, as all data that the
                // kernel before may have written) while the last product runs. The loops stay
                // rolled: this runs once per piece, so its instructions are fetched anew each time, and
                // unrolled it took 13,000 cycles per piece, most of them for that.
                const bool mine = r < rows, whole = w.whole(), gated = whole && a.gate != nullptr;
                const int row0 = w.t.row0 + PG_TOK * w.tile, h0 = KV_G * w.head;
                // box rows of PART dims, the 16-byte chunk c of row k at place c ^ (k / (128 / row bytes)): no
                // bank conflicts by rows nor by threads. Copy i of a lane: row RPC i + er, chunk ec.
                constexpr int PART = Fa<Q4>::PART, CH = PART / 8, RPC = 32 / CH, COPIES = 32 / RPC;
                const int er = lane / CH, ec = lane % CH;
                auto place = [&](int k, int c) { return k * PART * 2 + ((c ^ ((k * CH >> 3) & (CH - 1))) << 4); };
                unsigned char *box = blk + Fa<Q4>::EPI + (warp - 4) * Fa<Q4>::BOX;
                // row 32 q4 + k is token 4 q4 + k / 8, head k % 8
                uint4 gate[COPIES];
                const bf16 *gsrc = a.gate + (row0 + 4 * q4) * a.gate_row + (h0 + (er & 7)) * a.gate_head + 128 * grp + 8 * ec;
                auto load_gate = [&](int part) {
#pragma unroll
                    for (int i = 0; i < COPIES; ++i)
                        gate[i] = 4 * q4 + (RPC * i >> 3) < rows >> 3
                                      ? load_global(reinterpret_cast<const uint4 *>(gsrc + (RPC * i >> 3) * a.gate_row + (RPC * i & 7) * a.gate_head + PART * part))
                                      : make_uint4(0u, 0u, 0u, 0u);
                };
                if (gated && live) load_gate(0);
                reinterpret_cast<float *>(box)[lane] = l;      // the row's sum over both groups
                pair_bar();
                const float l1 = reinterpret_cast<const float *>(blk + Fa<Q4>::EPI + ((warp - 4) ^ 4) * Fa<Q4>::BOX)[lane];
                l = grp == 0 ? l + l1 : l1 + l;
                pair_bar2();
                ok = __all_sync(0xffffffffu, wait_pv(u - 1) && !aborted);
                tc::fence_after_sync();
                if (live && ok) {
                    if (__any_sync(0xffffffffu, *const_cast<const volatile int *>(&ss.poison) != 0)) {
                        // what the piece's value rows that not all see have left out
                        const int begin = max(max(all_see(), 0), w.unit * PG_TILE), end = min(limit_of(), (w.unit + w.len) * PG_TILE);
#pragma unroll 1
                        for (int d = 128 * grp; d < 128 * grp + 128; d += 16) {
                            uint32_t m = 0u, x[16];
#pragma unroll 1
                            for (int p = begin; p < end; ++p) m |= poison_of<Q4>(a, w.seq, w.head, p, d);
                            __syncwarp();              // the rows' ends differ
                            float o[16];
                            tc::tmem_ld16(lbase + FA_O + d, o);
                            tc::wait_ld();
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                x[k] = __float_as_uint(o[k] + ((m >> k & 1u) != 0u ? INFINITY : 0.0f) - ((m >> (16 + k) & 1u) != 0u ? INFINITY : 0.0f));
                            __syncwarp();
                            tc::tmem_st16_u32(lbase + FA_O + d, x);
                        }
                        tc::wait_st();
                    }
                }
                if (live && ok && !whole) {            // a piece: as it is, in fp32 (a row that saw nothing in it is left out by the join)
                    const size_t slot = ((size_t)2 * blockIdx.x + (w.first ? 0 : 1)) * a.rows + r;
#pragma unroll 1
                    for (int c = 128 * grp; c < 128 * grp + 128; c += 32) {
                        float o[32];
                        tc::tmem_ld32(lbase + FA_O + c, o);
                        tc::wait_ld();
                        if (mine)
#pragma unroll
                            for (int k = 0; k < 32; k += 4)
                                *reinterpret_cast<float4 *>(a.part_o + slot * KV_D + c + k) = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
                    }
                    if (mine && grp == 0) *reinterpret_cast<float2 *>(a.part_ml + slot * 2) = make_float2(m * SCORE_SCALE, l);
                } else if (live && ok) {
                    // a row that sees nothing gives zeros; one whose scores are all -infinity NaN, as the formula does
                    const bool blind = limit_of() <= 0, blank = __any_sync(0xffffffffu, blind);
                    const float inv = blind ? 0.0f : 1.0f / l;
                    TO *out = static_cast<TO *>(a.out);
#pragma unroll 1
                    for (int part = 0; part < 128 / PART; ++part) {
                        if (gated) {
#pragma unroll
                            for (int i = 0; i < COPIES; ++i) *reinterpret_cast<uint4 *>(box + place(RPC * i + er, ec)) = gate[i];
                            __syncwarp();
                            if (part + 1 < 128 / PART) load_gate(part + 1);
                        }
#pragma unroll 1
                        for (int c = 0; c < PART / 16; ++c) {  // 16 dims
                            const int d = 128 * grp + PART * part + 16 * c;
                            float o[16];
                            tc::tmem_ld16(lbase + FA_O + d, o);
                            uint4 *at[2], g[2];
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                at[i] = reinterpret_cast<uint4 *>(box + place(lane, 2 * c + i));
                                g[i] = gated ? *at[i] : make_uint4(0u, 0u, 0u, 0u);
                            }
                            tc::wait_ld();
                            if (blank)
#pragma unroll
                                for (int k = 0; k < 16; ++k) o[k] = blind ? 0.0f : o[k];
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                float e[8];
#pragma unroll
                                for (int k = 0; k < 8; ++k) e[k] = o[8 * i + k];
                                if (gated) {
                                    gate8(g[i], e, inv);
                                } else {
#pragma unroll
                                    for (int k = 0; k < 8; ++k) e[k] *= inv;
                                }
                                if (sizeof(TO) == 4) {
                                    if (mine) store8_out(out + ((size_t)(row0 + (r >> 3)) * KV_HQ + h0 + (r & 7)) * KV_D + d + 8 * i, e);
                                } else {
                                    store8_out(reinterpret_cast<bf16 *>(at[i]), e);
                                }
                            }
                            __syncwarp();
                        }
                        if (sizeof(TO) == 2) {
                            uint4 v[COPIES];
                            TO *dst = out + ((size_t)(row0 + 4 * q4) * KV_HQ + h0 + (er & 7)) * KV_D + 128 * grp + PART * part + 8 * ec;
#pragma unroll
                            for (int i = 0; i < COPIES; ++i) v[i] = *reinterpret_cast<const uint4 *>(box + place(RPC * i + er, ec));
#pragma unroll
                            for (int i = 0; i < COPIES; ++i)
                                if (4 * q4 + (RPC * i >> 3) < rows >> 3)
                                    *reinterpret_cast<uint4 *>(dst + ((RPC * i >> 3) * KV_HQ + (RPC * i & 7)) * KV_D) = v[i];
                            __syncwarp();
                        }
                    }
                }
                tc::fence_before_sync();
                mbar_arrive(smem_u32(&ss.o_empty));
                if (!ok || !w.more(a)) break;
                w.next(a);
            }
            if (!ok) {
                ss.top[0][grp][r] = ss.top[1][grp][r] = 0xFFFFFFFFu;
                ss.abort = 1;
                __threadfence_block();
                __syncwarp();
                asm volatile("bar.arrive %0, 64;\n\tbar.arrive %1, 64;" ::"r"(1 + q4), "r"(5 + q4) : "memory");
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 3) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tm, 512);
    }
    if (tid == 0 && ss.abort) atomicExch(&g_paged_error, (unsigned int)GDN_ERR_TIMEOUT);
}

// Joins the pieces of every item that spans ranges: with the pieces' maxima m_s
// (powers of two), sums l_s and unnormalised outputs o_s,
//   M = max m_s, out = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s * sigmoid(gate).
// There is one CTA for every cut between ranges and eight rows of an item. An item
// of n + 1 pieces has n cuts, so its CTAs, numbered over cuts and row groups, share
// its rows: eight to one each, as there are few or many pieces. The 8 warps of a CTA
// divide over its rows, those of a row over its pieces (8 dims per lane, four
// pieces' loads at a time), and meet in shared memory.
template <typename TO>
__global__ void __launch_bounds__(256) attn_paged_join_kernel(const PagedArgs a)
{
    __shared__ float so[8][KV_D], sml[8][2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x + 1;
    grid_dep_wait();
    grid_dep_launch();
    const PagedStart st = a.start[c];
    // the item's first step, and the step of its first unit: a cut at or before that one cuts nothing
    const long long u = range_begin(st, c), begin = u - st.step, unit0 = begin + a.lead;
    const long long total = range_begin(st, PG_RANGES);
    if (u >= total || u <= unit0) return;
    const SeqTokens t = st.t;
    const long long end = unit0 + tile_units(a, t, st.tile);
    // range_begin(k) is floor(total k / PG_RANGES): the first cut above unit0, and the last below end
    int head, last;
    if (total < 0xFFFFFFFFll / PG_RANGES) {
        head = (int)(((uint32_t)(unit0 + 1) * PG_RANGES + (uint32_t)total - 1) / (uint32_t)total);
        last = (int)(((uint32_t)end * PG_RANGES - 1) / (uint32_t)total);
    } else {
        head = (int)(((unit0 + 1) * PG_RANGES + total - 1) / total);
        last = (int)((end * PG_RANGES - 1) / total);
    }
    const int rows = KV_G * min(a.tok, t.n - (st.tile << a.tok_log2));
    const int ctas = (last - head + 1) * gridDim.y, cta = (c - head) * gridDim.y + blockIdx.y;
    int per = 1;                                       // rows of a CTA: a power of two up to 8
    while (per < 8 && per * ctas < rows) per <<= 1;
    const int share = 8 / per, r = cta * per + warp / share, part = warp % share;
    const int mrow = t.row0 + (st.tile << a.tok_log2) + (r >> 3), h = KV_G * st.head + (r & 7);
    uint4 gate = make_uint4(0u, 0u, 0u, 0u);
    const bool gated = a.gate != nullptr && r < rows && part == 0;
    if (gated) gate = *(reinterpret_cast<const uint4 *>(a.gate + mrow * a.gate_row + h * a.gate_head) + lane);
    float M = -INFINITY, l = 0.0f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int k0 = head - 1 + part; k0 <= last && r < rows; k0 += 4 * share) {
        float2 ml[4];
        float4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = k0 + share * i;
            ml[i] = make_float2(-INFINITY, 0.0f);
            x[i] = y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            const long long from = range_begin(st, k);
            if (k > last || range_begin(st, k + 1) == from) continue;   // past the item, or an empty range
            const size_t slot = ((size_t)2 * k + (from >= begin ? 0 : 1)) * a.rows + r;
            ml[i] = *reinterpret_cast<const float2 *>(a.part_ml + slot * 2);
            const float4 *src = reinterpret_cast<const float4 *>(a.part_o + slot * KV_D) + 2 * lane;
            x[i] = src[0];
            y[i] = src[1];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (ml[i].y == 0.0f) continue;             // a piece that saw nothing
            const float Mn = fmaxf(M, ml[i].x), f = ex2(M - Mn), g = ex2(ml[i].x - Mn);
            M = Mn;
            l = l * f + ml[i].y * g;
            o[0] = o[0] * f + x[i].x * g; o[1] = o[1] * f + x[i].y * g;
            o[2] = o[2] * f + x[i].z * g; o[3] = o[3] * f + x[i].w * g;
            o[4] = o[4] * f + y[i].x * g; o[5] = o[5] * f + y[i].y * g;
            o[6] = o[6] * f + y[i].z * g; o[7] = o[7] * f + y[i].w * g;
        }
    }
    if (share > 1) {                                   // the same for the whole CTA
        store8_out(&so[warp][8 * lane], o);
        if (lane == 0) {
            sml[warp][0] = M;
            sml[warp][1] = l;
        }
        __syncthreads();
        if (part != 0) return;
        for (int k = warp; k < warp + share; ++k) M = fmaxf(M, sml[k][0]);
        l = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = 0.0f;
        for (int k = warp; k < warp + share; ++k) {
            if (sml[k][1] == 0.0f) continue;
            const float g = ex2(sml[k][0] - M);
            l += g * sml[k][1];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] += g * so[k][8 * lane + i];
        }
    }
    if (r >= rows) return;
    // l is 0 where the row sees nothing (zeros), and where all its scores are -infinity (NaN, as the formula)
    const bool blind = t.first + (st.tile << a.tok_log2) + (r >> 3) < 0;
    const float inv = blind ? 0.0f : 1.0f / l;
    if (gated) gate8(gate, o, inv);
    else
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] *= inv;
    store8_out(static_cast<TO *>(a.out) + ((size_t)mrow * KV_HQ + h) * KV_D + 8 * lane, o);
}

// ------------------------------------------------------------------ launcher

// A tensor map with unit element strides and zero fill, through the driver's
// encoder (looked up once); false if that is missing or rejects the arguments.
bool encode_tiled(CUtensorMap *map, CUtensorMapDataType dt, int rank, const void *base, const cuuint64_t *dims,
                  const cuuint64_t *strides, const cuuint32_t *box, CUtensorMapSwizzle swizzle)
{
    typedef CUresult (*Fn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                           const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                           CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Fn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult r;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r);
        return e == cudaSuccess && r == cudaDriverEntryPointSuccess ? reinterpret_cast<Fn>(p) : nullptr;
    }();
    const cuuint32_t one[3] = {1, 1, 1};
    return fn && fn(map, dt, rank, const_cast<void *>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_paged_join(const PagedArgs &a, gdn_dtype out_dt, cudaStream_t s)
{
    const dim3 grid(PG_RANGES - 1, a.rows / KV_G), block(256);
    return out_dt == GDN_F32 ? launch_pdl(attn_paged_join_kernel<float>, grid, block, 0, s, a)
                             : launch_pdl(attn_paged_join_kernel<bf16>, grid, block, 0, s, a);
}

// [M][16][256] in boxes of 16 tokens x 8 heads x 64 dims, 128-byte swizzle; tokens past M read as zeros.
static bool encode_q_map(CUtensorMap *map, const void *q, int M)
{
    const cuuint64_t dims[3] = {KV_D, KV_HQ, (cuuint64_t)M}, strides[2] = {KV_D * 2, KV_HQ * KV_D * 2};
    const cuuint32_t box[3] = {64, KV_G, PG_TOK};
    return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, q, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// New tokens of a sequence up to which a 4-bit cache is read token by token: two take 271 us against 377 for a tile
// of all (76 contexts of 16,384), three 404 against 369; 64 contexts of 1,024: 31 against 36, 41 against 36.
constexpr int Q4_SINGLE = 2;
constexpr size_t START_BYTES = (PG_RANGES * sizeof(PagedStart) + 255) / 256 * 256;

static int piece_rows(int max_q) { return KV_G * (max_q < PG_TOK ? max_q : PG_TOK); }

size_t paged_workspace_bytes(const gdn_paged_batch *b, const gdn_kv_cache *)
{
    return START_BYTES + (size_t)2 * PG_RANGES * piece_rows(b->max_q) * (KV_D + 2) * sizeof(float);
}

template <typename TO, bool Q4>
static cudaError_t launch_tiles(const PagedArgs &a, cudaStream_t s)
{
    CUtensorMap qm, km = {}, vm = {};
    const long long rows = (long long)a.b.num_pages * KV_H * a.b.page;
    if (!encode_q_map(&qm, a.q, a.b.M) ||
        (!Q4 && (!make_bf16_sw128_map(&km, a.ck, rows, KV_D, a.b.page) || !make_bf16_sw128_map(&vm, a.cv, rows, KV_D, a.b.page))))
        return cudaErrorInvalidValue;
    const cudaError_t e = smem_attr_once<attn_paged_kernel<TO, Q4>>(FA_SMEM<Q4>);
    if (e != cudaSuccess) return e;
    return launch_pdl(attn_paged_kernel<TO, Q4>, dim3(PG_RANGES), dim3(fa_threads(Q4)), FA_SMEM<Q4>, s, qm, km, vm, a);
}

cudaError_t launch_attn_paged(const gdn_paged_batch *b, const gdn_kv_cache *c, const void *q, const void *gate,
                              long long gate_row, long long gate_head, void *out, void *ws, gdn_dtype out_dt,
                              cudaStream_t s)
{
    PagedArgs a = {};
    a.b = paged_batch(*b, *c);
    a.ck = c->k;
    a.cv = c->v;
    a.q = (const bf16 *)q;
    a.gate = (const bf16 *)gate;
    a.gate_row = gate_row;
    a.gate_head = gate_head;
    a.out = out;
    a.rows = piece_rows(b->max_q);
    // an item's own cost in units of tiles. One prompt of 4,096: 174 us with 2, 150 with 3, 139 with 4, 140 with
    // 6, 144 with 8. Items of fewer rows have a shorter epilogue and tiles bound by HBM, and it matters little:
    // with 1, 2, 3 and 4, four tokens on 64 contexts of 2,048 take 54, 57, 57 and 56 us, eight on 20 of 4,096 44, 43,
    // 44 and 43, one token on 256 of 2,048 166, 165, 166 and 166; over 4-bit pages 78, 78, 77 and 78
    a.tok = PG_TOK;
    a.tok_log2 = 4;
    a.lead = b->max_q >= PG_TOK ? 4 : b->max_q > 1 ? 3 : 2;
    a.start = (PagedStart *)ws;
    a.part_o = (float *)((char *)ws + START_BYTES);
    a.part_ml = a.part_o + (size_t)2 * PG_RANGES * a.rows * KV_D;
    cudaError_t e;
    if (c->format == GDN_KV_Q4 && b->max_q <= Q4_SINGLE) {
        a.tok = 1;
        a.tok_log2 = 0;
        a.rows = KV_G;
        a.lead = 2;
        e = launch_paged_q4(a, out_dt, s);
    } else if (c->format == GDN_KV_Q4) {
        e = out_dt == GDN_F32 ? launch_tiles<float, true>(a, s) : launch_tiles<bf16, true>(a, s);
    } else {
        e = out_dt == GDN_F32 ? launch_tiles<float, false>(a, s) : launch_tiles<bf16, false>(a, s);
    }
    return e == cudaSuccess ? launch_paged_join(a, out_dt, s) : e;
}

// Device address of this file's error word, for gdn_device_error.
void *paged_error_word()
{
    void *p = nullptr;
    return cudaGetSymbolAddress(&p, g_paged_error) == cudaSuccess ? p : nullptr;
}

}  // namespace gdn
