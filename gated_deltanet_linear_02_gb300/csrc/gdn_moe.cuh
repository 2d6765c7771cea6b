// gdn_moe.cuh -- what the kernels of the mixture-of-experts layer share: the
// workspace of one call, and tensor-core and copy forms that only they use.
#pragma once

#include <cuda_fp16.h>

#include "gdn_layer.cuh"

namespace gdn {

constexpr int MOE_WINDOW = 8192;          // tokens that one pass over the experts takes, at most
constexpr int MOE_TILE = 128;             // tokens of one product, at most
// Tokens per expert, for even routing, up to which tiles hold 32 and y is fp32. 8 of 256 experts: 384 tokens 274 us
// with tiles of 32 and 274 of 128, 512 tokens 285 and 278, 640 tokens 297 and 282, 1,024 tokens 347 and 291.
constexpr int MOE_SMALL = 16;
constexpr int MOE_ROUTE_TILE = 128;       // tokens of a cluster of the router
// Tokens up to which the weights pass through the CUDA cores. 8 of 256 experts: 2 tokens 32.7 us there and 43.7
// through the tensor cores, 4 tokens 52.9 and 53.5, 5 tokens 63.8 and 62.5, 8 tokens 104 and 73.6.
constexpr int MOE_FEW_TOKENS = 4;

// A 2-D box (gdn_tma.cuh) that leaves L2 before what is read again.
__device__ __forceinline__ uint64_t evict_first_policy()
{
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ void tma_load_2d_hint(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar, uint64_t policy)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
                 "[%0], [%1, {%2, %3}], [%4], %5;"
                 ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "l"(policy) : "memory");
}

// Four rows y of a row-major matrix, 64 columns from x on, to four consecutive
// 128-byte rows of shared memory (tensor map of 64 x 1 boxes, 128-byte swizzle).
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap *map, int x, int4 y, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];"
                 ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w),
                   "r"(bar) : "memory");
}

// Where the pairs (token, expert) go: each expert's list of tokens, in any order (a
// token's result does not depend on its place), filled through counters.
struct MoePlaces {
    int *count;                           // [E], zero before the first pair; NULL: no places wanted
    int *token;                           // [E][stride]
    int *rank;                            // [tokens][k]: the pair's place in its expert's list, or -1
    int stride;                           // tokens * k: a given routing may name an expert several times a token
};

__device__ __forceinline__ void place_pair(const MoePlaces &p, int m, int slot, int e, int k)
{
    const int r = atomicAdd(p.count + e, 1);
    p.token[(size_t)e * p.stride + r] = m;
    p.rank[(size_t)m * k + slot] = r;
}

// Workspace of a window of at most W tokens. Rows of h and y: each expert's pairs in
// the order of its list, one expert after the other, then the shared expert's, in
// token order, from row W * top_k on.
struct MoeWs {
    int *state;                           // what a call starts from zero: ticket, count, ready
    size_t state_ints;
    int *ticket;                          // next unit of work
    int *ready;                           // [tiles] finished parts of each tile's h
    int *offset;                          // [E] first row of each expert
    MoePlaces places;
    int *ids;
    float *weights;
    bf16 *h;                              // [rows][F]
    float *y;                             // [rows][2048] outputs of the pairs. Few tokens: h in fp32, [rows][F];
                                          // many: y16 and scale in its place
    __half *y16;                          // [rows][2048], scaled by blocks of 32
    unsigned char *scale;                 // [rows][64]: y = y16 * 2^(scale - 141)
    float *logits;                        // few tokens: [M][E + 1], and their sums of magnitudes
    size_t bytes;
};

inline bool moe_small(const gdn_moe_params *p, int M)
{
    return (long long)M * p->top_k <= (long long)MOE_SMALL * p->num_experts;
}

inline int moe_max_tiles(const gdn_moe_params *p, int W)
{
    const long long pairs = (long long)W * p->top_k;
    const int e = (int)(pairs < p->num_experts ? pairs : p->num_experts);
    return (int)(pairs / 16) + e + W / 16 + 2;    // tiles of 16 tokens and more; the last of each expert may be partial
}

inline MoeWs moe_workspace(const gdn_moe_params *p, int M, void *base)
{
    const int W = M < MOE_WINDOW ? M : MOE_WINDOW;
    const bool shared = p->sh_gate != nullptr;
    const size_t pairs = (size_t)W * p->top_k, rows = pairs + (shared ? W : 0);
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t here = at;
        at += (n + 255) & ~(size_t)255;
        return static_cast<char *>(base) + here;
    };
    const int tiles = moe_max_tiles(p, W);
    MoeWs w;
    w.state_ints = 1 + GDN_MOE_MAX_EXPERTS + (size_t)tiles;   // few tokens: two counters
    w.state = (int *)take(w.state_ints * 4);
    w.ticket = w.state;
    w.places.count = w.state + 1;
    w.ready = w.state + 1 + GDN_MOE_MAX_EXPERTS;
    w.offset = (int *)take(GDN_MOE_MAX_EXPERTS * 4);
    w.places.token = (int *)take((size_t)p->num_experts * pairs * 4);
    w.places.rank = (int *)take(pairs * 4);
    w.places.stride = (int)pairs;
    w.ids = (int *)take(pairs * 4);
    w.weights = (float *)take(pairs * 4);
    w.h = (bf16 *)take(rows * p->ffn_dim * 2);
    const size_t y_row = W > MOE_FEW_TOKENS && !moe_small(p, M) ? LD * 2 + LD / 32 : (size_t)(W <= MOE_FEW_TOKENS && p->ffn_dim > LD ? p->ffn_dim : LD) * 4;
    w.y = (float *)take(rows * y_row);
    w.y16 = reinterpret_cast<__half *>(w.y);
    w.scale = reinterpret_cast<unsigned char *>(w.y) + rows * LD * 2;
    w.logits = (float *)take(W <= MOE_FEW_TOKENS ? (size_t)W * (p->num_experts + 1) * 8 : 0);
    w.bytes = at;
    return w;
}

cudaError_t launch_route(const gdn_moe_params *p, const void *x, long long x_row, int M, int32_t *ids, float *weights,
                         const MoePlaces &places, int *state, int n_state, bool lose, cudaStream_t s);

cudaError_t launch_moe_few(const gdn_moe_params *p, const void *x, long long x_row, const void *residual, void *out, int M,
                           const int32_t *ids, const float *weights, const MoeWs &ws, gdn_dtype out_dt, cudaStream_t s);

}  // namespace gdn
