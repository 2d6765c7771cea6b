// gdn_route.cuh -- a warp's choice of the top_k experts of one token, from logits
// that it holds 8 a lane (gdn_route.cu for many tokens, gdn_moe_few.cu for few).
#pragma once

#include "gdn_layer.cuh"

namespace gdn {

constexpr int RT_MAX_E = GDN_MOE_MAX_EXPERTS;
constexpr int RT_SLOTS = RT_MAX_E / 32;   // logits per lane

// A lane holds experts 4 lane .. 4 lane + 3 (slots 0 to 3) and 128 + 4 lane .. (slots 4 to 7), so
// that logits come 16 bytes at a time. A larger slot is a larger expert.
static_assert(RT_SLOTS == 8, "two vectors of four logits a lane");
__device__ __forceinline__ int expert_of(int lane, int j) { return (j >> 2) * 128 + lane * 4 + (j & 3); }
__device__ __forceinline__ int lane_of(int e) { return (e >> 2) & 31; }
__device__ __forceinline__ int slot_of(int e) { return (e >> 7) * 4 + (e & 3); }

// Order-preserving keys of floats; NaN is the smallest, -0 is +0.
__device__ __forceinline__ uint32_t sort_key(float x)
{
    if (!(x == x)) return 0u;
    const uint32_t u = __float_as_uint(x + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// a + b as (sum, error), both exact.
__device__ __forceinline__ float2 two_sum(float a, float b)
{
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return make_float2(s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t)));
}
__device__ __forceinline__ float2 pair_add(float2 a, float2 b)
{
    const float2 s = two_sum(a.x, b.x);
    const float e = __fadd_rn(s.y, __fadd_rn(a.y, b.y)), h = __fadd_rn(s.x, e);
    return make_float2(h, __fsub_rn(e, __fsub_rn(h, s.x)));
}

// The logit of one expert as a pair of fp32, the same in every lane. Four running
// sums, each with the sum of its rounding errors beside it: one addition per product
// on the critical path.
static __device__ __noinline__ float2 pair_dot(const bf16 *x, const bf16 *w, int lane)
{
    float2 acc[4] = {};
    uint4 xs[LD / 256], ws[LD / 256];                  // all loads in flight together
#pragma unroll
    for (int c = 0; c < LD / 256; ++c) {
        ws[c] = *reinterpret_cast<const uint4 *>(w + c * 256 + lane * 8);
        xs[c] = *reinterpret_cast<const uint4 *>(x + c * 256 + lane * 8);
    }
#pragma unroll
    for (int c = 0; c < LD / 256; ++c) {
        float a[8], b[8];
        unpack8(xs[c], a);
        unpack8(ws[c], b);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 s = two_sum(acc[i & 3].x, __fmul_rn(a[i], b[i]));
            acc[i & 3] = make_float2(s.x, __fadd_rn(acc[i & 3].y, s.y));
        }
    }
    float2 sum = pair_add(pair_add(acc[0], acc[1]), pair_add(acc[2], acc[3]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        sum = pair_add(sum, make_float2(__shfl_xor_sync(0xffffffffu, sum.x, o), __shfl_xor_sync(0xffffffffu, sum.y, o)));
    return sum;
}

// The same choice as below for tokens where dozens of logits are near one another.
static __device__ __noinline__ void choose_settled(const float *logits, int E, int k, bool renorm, float tie, const bf16 *x,
                                                   const bf16 *router, int lane, int &id, float &weight)
{
    uint32_t key[RT_SLOTS];
    float v[RT_SLOTS];
#pragma unroll
    for (int j = 0; j < RT_SLOTS; ++j) v[j] = logits[j];
#pragma unroll
    for (int j = 0; j < RT_SLOTS; ++j) key[j] = expert_of(lane, j) < E ? sort_key(v[j]) : 0u;
    float lo[RT_SLOTS];
#pragma unroll
    for (int j = 0; j < RT_SLOTS; ++j) lo[j] = 0.0f;
    float best = 0.0f;                                 // lane i: the i-th logit
    id = 0;
    bool settled = false;
    for (;;) {
        uint32_t taken = 0;                            // this lane's slots that are out
        uint32_t near = 0;                             // this lane's slots that are close to a neighbour
        float prev = 0.0f, kth = 0.0f;
        int prev_at = 0;
        bool close = false, border = false;
        const int rounds = settled || k >= E ? k : k + 1;
        for (int i = 0; i < rounds; ++i) {
            uint32_t mk = 0;
#pragma unroll
            for (int j = 0; j < RT_SLOTS; ++j)
                if (!(taken >> j & 1u) && expert_of(lane, j) < E) mk = max(mk, key[j]);
            const uint32_t top = __reduce_max_sync(0xffffffffu, mk);
            uint32_t ml = 0;                           // settled: the larger low part among equal high ones
            if (settled) {
#pragma unroll
                for (int j = 0; j < RT_SLOTS; ++j)
                    if (!(taken >> j & 1u) && expert_of(lane, j) < E && key[j] == top) ml = max(ml, sort_key(lo[j]));
                ml = __reduce_max_sync(0xffffffffu, ml);
            }
            uint32_t at = 0xffffffffu;
#pragma unroll
            for (int j = RT_SLOTS - 1; j >= 0; --j)
                if (!(taken >> j & 1u) && expert_of(lane, j) < E && key[j] == top && (!settled || sort_key(lo[j]) == ml))
                    at = (uint32_t)expert_of(lane, j);
            at = __reduce_min_sync(0xffffffffu, at);
            float val = 0.0f;
#pragma unroll
            for (int j = 0; j < RT_SLOTS; ++j)
                if ((int)at == expert_of(lane, j)) {
                    val = v[j];
                    taken |= 1u << j;
                }
            val = __shfl_sync(0xffffffffu, val, lane_of((int)at));
            if (i > 0 && prev - val <= tie) {
                close = true;
                border |= i == k;
                if (lane_of(prev_at) == lane) near |= 1u << slot_of(prev_at);
                if (lane_of((int)at) == lane) near |= 1u << slot_of((int)at);
            }
            prev = val;
            prev_at = (int)at;
            if (i < k) {
                kth = val;
                if (lane == i) {
                    best = val;
                    id = (int)at;
                }
            }
        }
        if (settled || !close || !(tie > 0.0f)) break;
        // in 48 bits: the neighbours among the first k, and where the last of them is
        // close to the next, every expert that may be in its place
        settled = true;
        if (border) {
#pragma unroll
            for (int j = 0; j < RT_SLOTS; ++j)
                if (expert_of(lane, j) < E && !(v[j] < kth - tie) && v[j] <= kth) near |= 1u << j;
        }
#pragma unroll
        for (int j = 0; j < RT_SLOTS; ++j) {
            uint32_t who = __ballot_sync(0xffffffffu, (near >> j & 1u) && fabsf(v[j]) < INFINITY);
            while (who) {
                const int from = __ffs(who) - 1;
                who &= who - 1;
                const float2 p = pair_dot(x, router + (size_t)expert_of(from, j) * LD, lane);
                if (lane == from) {
                    v[j] = p.x;
                    key[j] = sort_key(p.x);
                    lo[j] = p.y;
                }
            }
        }
    }
    const float top = __shfl_sync(0xffffffffu, best, 0);
    const float ex = lane < k ? expf(best - top) : 0.0f;
    float sum = ex;
    if (!renorm) {
        sum = 0.0f;
#pragma unroll
        for (int j = 0; j < RT_SLOTS; ++j)
            if (expert_of(lane, j) < E) sum += expf(v[j] - top);
    }
    weight = ex / warp_sum(sum);
}

// The k largest of the warp's logits v[j] (expert_of(lane, j); whatever past E):
// lane i < k gets the i-th expert and its weight. `tie` bounds how far the difference of two of
// these logits is from the exact one, so that closer ones may be in the wrong order; it follows
// the sums of magnitudes that the logits are sums of, which may be any multiple of the
// logits themselves. 0: all logits are 0 or not finite, nothing is to be settled.
__device__ __forceinline__ void choose(const float (&v)[RT_SLOTS], int E, int k, bool renorm, float tie, const bf16 *x,
                                       const bf16 *router, int lane, int &id, float &weight)
{
    uint32_t key[RT_SLOTS];
#pragma unroll
    for (int j = 0; j < RT_SLOTS; ++j) key[j] = expert_of(lane, j) < E ? sort_key(v[j]) : 0u;
    // the largest k, and behind them those that are close to the last of them; a lane
    // offers the best that it has left, lane i keeps the i-th
    float best = 0.0f, prev = 0.0f, kth = -INFINITY;
    bool close = false;
    id = 0;
    uint32_t left = 0;                                 // this lane's slots below E
#pragma unroll
    for (int j = 0; j < RT_SLOTS; ++j) left |= (uint32_t)(expert_of(lane, j) < E) << j;
    const int most = min(E, 32);
    int n = 0;
#pragma unroll 1
    for (; n < most; ++n) {
        uint32_t mk = 0, mj = 0;
#pragma unroll
        for (int j = RT_SLOTS - 1; j >= 0; --j)
            if ((left >> j & 1u) && key[j] >= mk) {
                mk = key[j];
                mj = (uint32_t)j;
            }
        const uint32_t top = __reduce_max_sync(0xffffffffu, mk);
        const uint32_t at = __reduce_min_sync(0xffffffffu, left != 0u && mk == top ? (uint32_t)expert_of(lane, (int)mj) : 0xffffffffu);
        const float val = top == 0u ? __uint_as_float(0x7fffffffu) : __uint_as_float((top & 0x80000000u) ? top ^ 0x80000000u : ~top);
        if (n >= k && !(kth - val <= tie)) break;
        if (lane_of((int)at) == lane) left &= ~(1u << slot_of((int)at));
        close |= n > 0 && prev - val <= tie;
        prev = val;
        if (n < k) kth = val;
        if (lane == n) {
            best = val;
            id = (int)at;
        }
    }
    if (close && tie > 0.0f) {
        if (n == 32 && E > 32) {                       // more neighbours than lanes
            choose_settled(v, E, k, renorm, tie, x, router, lane, id, weight);
            return;
        }
        // in 48 bits those that are close to a neighbour, then every one's place among the n
        const float up = __shfl_up_sync(0xffffffffu, best, 1), down = __shfl_down_sync(0xffffffffu, best, 1);
        const bool near = lane < n && fabsf(best) < INFINITY && ((lane > 0 && up - best <= tie) || (lane + 1 < n && best - down <= tie));
        float low = 0.0f;
        for (uint32_t who = __ballot_sync(0xffffffffu, near); who; who &= who - 1)     // their rows, all at once
            asm volatile("prefetch.global.L1 [%0];" ::"l"(router + (size_t)__shfl_sync(0xffffffffu, id, __ffs(who) - 1) * LD + lane * 64));
        for (uint32_t who = __ballot_sync(0xffffffffu, near); who; who &= who - 1) {
            const int from = __ffs(who) - 1;
            const float2 p = pair_dot(x, router + (size_t)__shfl_sync(0xffffffffu, id, from) * LD, lane);
            if (lane == from) {
                best = p.x;
                low = p.y;
            }
        }
        const uint32_t mine = sort_key(best);
        int place = 0;
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
            const uint32_t kj = __shfl_sync(0xffffffffu, mine, j);
            const float lj = __shfl_sync(0xffffffffu, low, j);
            const int ej = __shfl_sync(0xffffffffu, id, j);
            place += kj > mine || (kj == mine && (lj > low || (lj == low && ej < id)));
        }
        int from = 0;
#pragma unroll 1
        for (int j = 0; j < n; ++j)
            if (__shfl_sync(0xffffffffu, place, j) == lane) from = j;
        best = __shfl_sync(0xffffffffu, best, from);
        id = __shfl_sync(0xffffffffu, id, from);
    }
    const float top = __shfl_sync(0xffffffffu, best, 0);
    const float ex = lane < k ? expf(best - top) : 0.0f;
    float sum = ex;
    if (!renorm) {
        sum = 0.0f;
#pragma unroll 1
        for (int j = 0; j < RT_SLOTS; ++j)
            if (expert_of(lane, j) < E) sum += expf(v[j] - top);
    }
    weight = ex / warp_sum(sum);
}

}  // namespace gdn
