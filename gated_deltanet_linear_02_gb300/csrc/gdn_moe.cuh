// gdn_moe.cuh -- what the kernels of the mixture-of-experts layer share: the
// workspace of one call, and tensor-core and copy forms that only they use.
#pragma once

#include "gdn_layer.cuh"

namespace gdn {

constexpr int MOE_WINDOW = 8192;          // tokens that one pass over the experts takes, at most
constexpr int MOE_TILE = 128;             // tokens of one product, at most

__device__ __forceinline__ float ld_cluster_f32(uint32_t cluster_addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
    return v;
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

// Workspace of a window of at most W tokens: routing, the pairs (token, expert)
// sorted by expert, their activations h and their outputs y. The shared expert's
// rows follow the W * top_k routed ones, in token order.
struct MoeWs {
    int *ticket;                          // next unit of work
    int *count, *offset;                  // [E] pairs of each expert, and where they begin
    int *ready;                           // [tiles] finished parts of each tile's h
    int *token, *place;                   // sorted pair -> token; (token, slot) -> sorted pair, or -1
    int *ids;
    float *weights;
    bf16 *h;                              // [rows][F]
    float *y;                             // [rows][2048]
    size_t bytes;
};

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
    MoeWs w;
    w.ticket = (int *)take(4);
    w.count = (int *)take(GDN_MOE_MAX_EXPERTS * 4);
    w.offset = (int *)take(GDN_MOE_MAX_EXPERTS * 4);
    w.ready = (int *)take((size_t)moe_max_tiles(p, W) * 4);
    w.token = (int *)take(pairs * 4);
    w.place = (int *)take(pairs * 4);
    w.ids = (int *)take(pairs * 4);
    w.weights = (float *)take(pairs * 4);
    w.h = (bf16 *)take(rows * p->ffn_dim * 2);
    w.y = (float *)take(rows * LD * 4);
    w.bytes = at;
    return w;
}

cudaError_t launch_route(const gdn_moe_params *p, const void *x, long long x_row, int M, int32_t *ids, float *weights,
                         cudaStream_t s);

}  // namespace gdn
