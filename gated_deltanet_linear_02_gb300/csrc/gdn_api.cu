// gdn_api.cu -- the C ABI declared in include/gdn.h: argument checks and
// dispatch to the kernels. Nothing here allocates or synchronises (except
// gdn_device_error, which is documented to).
#include <stdio.h>
#include <string.h>

#include <mutex>

#include "gdn_common.cuh"

namespace gdn {
void *decode_error_word();
cudaError_t launch_conv_step(const float *, const void *, void *, void *, int, gdn_dtype, cudaStream_t);
cudaError_t launch_decode_step(const gdn_params *, const void *, const void *, const void *, const void *,
                               void *, float *, void *, int, gdn_dtype, gdn_dtype, cudaStream_t);
cudaError_t launch_decode_multi(const gdn_params *, const void *, const void *, const void *, const void *,
                                void *, float *, void *, int, int, gdn_dtype, gdn_dtype, cudaStream_t);
void *multi_error_word();
cudaError_t launch_out_proj(const void *x, const void *w, void *y, int M, gdn_dtype out_dt, cudaStream_t s);
void *gemm_error_word();
cudaError_t launch_gated_out_proj(const float *norm_w, float eps, const void *y, const void *z, const void *w,
                                  void *out, int M, gdn_dtype act, gdn_dtype out_dt, cudaStream_t s);
void *gproj_error_word();
cudaError_t launch_in_proj(const void *h, const void *w_in, void *qkv, void *z, void *alpha, void *beta, int M,
                           gdn_dtype act, cudaStream_t s);
size_t scan_workspace_bytes(int T_total);
cudaError_t launch_prefill_scan(const gdn_params *, const void *, const void *, const void *, const void *,
                                const int32_t *, int, int, const void *, void *, const float *, float *,
                                void *, gdn_dtype, gdn_dtype, void *, cudaStream_t);
size_t chunk_workspace_bytes(int N, int T_total);
size_t chunk_min_workspace_bytes(int N);
cudaError_t launch_prefill_chunked(const gdn_params *, const void *, const void *, const void *, const void *,
                                   const int32_t *, int, int, const void *, void *, const float *, float *, void *,
                                   gdn_dtype, void *, size_t, cudaStream_t, const void *xhat_ext);
void *chunk_error_word();
cudaError_t launch_in_proj_conv(const float *conv_w, float l2_eps, const void *h, const void *w_in,
                                const int32_t *cu, int N, int M, const void *cs_in, void *cs_out, void *xhat,
                                void *z, void *alpha, void *beta, cudaStream_t s);
void *inconv_error_word();
size_t attn_workspace_bytes(int B, int Lmax);
cudaError_t launch_attn_decode(const void *q, const void *k_cache, const void *v_cache, const int32_t *ctx_len,
                               const void *z, void *out, int B, int Lmax, void *ws, gdn_dtype out_dt,
                               cudaStream_t s);
void *attn_error_word();
cudaError_t launch_qk_norm_rope(const gdn_attn_params *p, const void *q, long long q_row, long long q_head,
                                const void *k, long long k_row, long long k_head, const int32_t *positions, int M,
                                void *q_out, void *k_out, gdn_dtype act, gdn_dtype out_dt, cudaStream_t s);
cudaError_t launch_kv_append(const gdn_attn_params *p, const gdn_paged_batch *b, const gdn_kv_cache *c, const void *k,
                             long long k_row, long long k_head, const void *v, long long v_row, long long v_head,
                             const void *q, long long q_row, long long q_head, void *q_out, const int32_t *positions,
                             gdn_dtype act, cudaStream_t s);
cudaError_t launch_kv_gather(const gdn_paged_batch *b, const gdn_kv_cache *c, void *k_out, void *v_out,
                             gdn_dtype out_dt, cudaStream_t s);
void *paged_error_word();
void *paged_q4_error_word();
size_t paged_workspace_bytes(const gdn_paged_batch *b, const gdn_kv_cache *c);
cudaError_t launch_attn_paged(const gdn_paged_batch *b, const gdn_kv_cache *c, const void *q, const void *gate,
                              long long gate_row, long long gate_head, void *out, void *ws, gdn_dtype out_dt,
                              cudaStream_t s);
cudaError_t launch_add_norm(const gdn_norm_params *, const void *, long long, const void *, long long, const void *,
                            long long, void *, long long, void *, long long, int, gdn_dtype, gdn_dtype, cudaStream_t);
cudaError_t launch_linear(const void *, long long, const void *, const float *, const void *, long long, void *,
                          long long, int, int, int, gdn_activation, gdn_dtype, cudaStream_t);
void *linear_error_word();
cudaError_t launch_route_only(const gdn_moe_params *, const void *, long long, int, int32_t *, float *, cudaStream_t);
void *route_error_word();
size_t moe_workspace_bytes(const gdn_moe_params *, int), moe_call_bytes(const gdn_moe_params *, int);
cudaError_t launch_moe(const gdn_moe_params *, const void *, long long, const void *, void *, int, const int32_t *,
                       const float *, void *, gdn_dtype, bool, cudaStream_t);
void *moe_error_word();
void *few_error_word();
cudaError_t launch_wait_timeout(cudaStream_t s);
void *selftest_error_word();
}  // namespace gdn

using namespace gdn;

namespace {

thread_local char g_last_error[256] = "";

gdn_status fail(gdn_status s, const char *what)
{
    snprintf(g_last_error, sizeof(g_last_error), "%s", what);
    return s;
}

gdn_status cuda_fail(cudaError_t e, const char *where)
{
    snprintf(g_last_error, sizeof(g_last_error), "%s: %s", where, cudaGetErrorString(e));
    return GDN_ERR_CUDA;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool ok_ptr(const void *p) { return p != nullptr && aligned16(p); }
bool ok_opt_ptr(const void *p) { return p == nullptr || aligned16(p); }
bool ok_dtype(gdn_dtype d) { return d == GDN_F32 || d == GDN_BF16; }

gdn_status check_params(const gdn_params *p)
{
    if (p == nullptr) return fail(GDN_ERR_INVALID_ARG, "params is NULL");
    if (!ok_ptr(p->conv_w) || !ok_ptr(p->A_log) || !ok_ptr(p->dt_bias) || !ok_opt_ptr(p->norm_w))
        return fail(GDN_ERR_INVALID_ARG, "a parameter pointer is NULL or not 16-byte aligned");
    if (!(p->norm_eps >= 0.0f) || !(p->l2_eps >= 0.0f))
        return fail(GDN_ERR_INVALID_ARG, "epsilons must be >= 0");
    return GDN_OK;
}

constexpr int MAX_B = 65535;
constexpr int MAX_N = 65535;
constexpr int MAX_T = 1 << 24;
constexpr size_t WS_HEADER = 256;   // keeps the workspace body 256-byte aligned

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Do [a, a + an) and [b, b + bn) share a byte?
bool overlap(const void *a, size_t an, const void *b, size_t bn)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return an > 0 && bn > 0 && x < y + bn && y < x + an;
}

// A head tensor [M][heads][256] with element strides: the strides keep every row
// 16-byte aligned, and rows and heads do not run into each other.
struct Heads {
    const void *p;
    long long row, head;
    int heads;
    gdn_dtype dt;
    size_t bytes(int M) const
    {
        return ((size_t)(M - 1) * (size_t)row + (size_t)(heads - 1) * (size_t)head + GDN_ATTN_HEAD_DIM) *
               (dt == GDN_F32 ? 4 : 2);
    }
    bool dense() const { return head == GDN_ATTN_HEAD_DIM && row == (long long)heads * GDN_ATTN_HEAD_DIM; }
};
gdn_status check_heads(const Heads &t)
{
    const long long q = t.dt == GDN_F32 ? 4 : 8;
    if (!ok_ptr(t.p)) return fail(GDN_ERR_INVALID_ARG, "a tensor pointer is NULL or not 16-byte aligned");
    if (t.head < GDN_ATTN_HEAD_DIM || t.row < 0 || t.row % q || t.head % q || t.row > (1ll << 32) ||
        t.head > (1ll << 32))
        return fail(GDN_ERR_INVALID_ARG, "a stride is negative, below the head dim, above 2^32 or not a multiple of 16 bytes");
    return GDN_OK;
}

gdn_status check_attn_params(const gdn_attn_params *p)
{
    if (p == nullptr) return fail(GDN_ERR_INVALID_ARG, "attention params is NULL");
    if (!ok_opt_ptr(p->q_norm_w) || !ok_opt_ptr(p->k_norm_w) || !ok_opt_ptr(p->rope))
        return fail(GDN_ERR_INVALID_ARG, "a parameter pointer is not 16-byte aligned");
    if (!(p->norm_eps >= 0.0f)) return fail(GDN_ERR_INVALID_ARG, "norm_eps must be >= 0");
    if (p->rope != nullptr && p->n_pos < 1) return fail(GDN_ERR_INVALID_ARG, "n_pos must be >= 1 with a rotation table");
    return GDN_OK;
}

size_t kv_cache_bytes(const gdn_kv_cache *c)
{
    const size_t rows = (size_t)c->num_pages * GDN_ATTN_KV_HEADS * (size_t)c->page_size;
    return c->format == GDN_KV_Q4 ? rows / GDN_KV_RECORD_ROWS * GDN_KV_RECORD_BYTES : rows * GDN_ATTN_HEAD_DIM * 2;
}

gdn_status check_batch_sizes(const gdn_paged_batch *b, const gdn_kv_cache *c)
{
    if (b == nullptr || c == nullptr) return fail(GDN_ERR_INVALID_ARG, "batch or cache is NULL");
    if (c->format != GDN_KV_BF16 && c->format != GDN_KV_Q4) return fail(GDN_ERR_INVALID_ARG, "unknown cache format");
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
        return fail(GDN_ERR_INVALID_ARG, "page_size must be 16, 32, 64 or 128");
    if (c->num_pages < 1 || (long long)c->num_pages * GDN_ATTN_KV_HEADS * c->page_size > (1ll << 30))
        return fail(GDN_ERR_INVALID_ARG, "num_pages out of range: need 1 <= num_pages and num_pages * 2 * page_size <= 2^30");
    if (b->B < 0 || b->B > MAX_B) return fail(GDN_ERR_INVALID_ARG, "B out of range [0, 65535]");
    if (b->M < 0 || b->M > MAX_T) return fail(GDN_ERR_INVALID_ARG, "M out of range [0, 2^24]");
    if (b->max_pages < 1 || (long long)b->max_pages * c->page_size > (1ll << 30))
        return fail(GDN_ERR_INVALID_ARG, "max_pages out of range: need 1 <= max_pages and max_pages * page_size <= 2^30");
    if (b->cu_q == nullptr && (b->max_q != 1 || b->M < b->B))
        return fail(GDN_ERR_INVALID_ARG, "without cu_q, max_q must be 1 and M at least B");
    if (b->max_q < 1 || b->max_q > MAX_T) return fail(GDN_ERR_INVALID_ARG, "max_q out of range [1, 2^24]");
    return GDN_OK;
}

gdn_status check_batch(const gdn_paged_batch *b, const gdn_kv_cache *c)
{
    const gdn_status st = check_batch_sizes(b, c);
    if (st != GDN_OK || b->B == 0 || b->M == 0) return st;
    if (!ok_ptr(c->k) || (c->format == GDN_KV_BF16 && !ok_ptr(c->v)) || (c->format == GDN_KV_Q4 && c->v != nullptr))
        return fail(GDN_ERR_INVALID_ARG, "a cache pointer is NULL or not 16-byte aligned, or a 4-bit cache has a v");
    if (!b->page_table || !b->ctx_len || !aligned4(b->page_table) || !aligned4(b->ctx_len) || !aligned4(b->cu_q))
        return fail(GDN_ERR_INVALID_ARG, "page_table, ctx_len or cu_q is NULL or not 4-byte aligned");
    return GDN_OK;
}

size_t elem_size(gdn_dtype d) { return d == GDN_F32 ? 4 : 2; }

// Rows of `width` elements, `row` elements apart: how far they reach, and whether
// the stride keeps them 16-byte aligned and apart (0, one row for all, where `once`).
struct Rows {
    const void *p;
    long long row;
    int width;
    gdn_dtype dt;
    size_t bytes(int M) const { return ((size_t)(M - 1) * (size_t)row + (size_t)width) * elem_size(dt); }
    bool ok(bool once = false) const
    {
        return ok_ptr(p) && row % (long long)(16 / elem_size(dt)) == 0 && row <= (1ll << 32) &&
               (row >= width || (once && row == 0));
    }
};
// Whether M rows of each share an element. Rows the same distance apart (blocks of columns of one
// buffer) do not where each block ends before the other's next row begins; others
// count as overlapping where their address ranges do.
bool overlap(const Rows &a, const Rows &b, int M)
{
    if (!a.p || !b.p || !overlap(a.p, a.bytes(M), b.p, b.bytes(M))) return false;
    const size_t step = (size_t)a.row * elem_size(a.dt), wa = (size_t)a.width * elem_size(a.dt),
                 wb = (size_t)b.width * elem_size(b.dt);
    if (M == 1 || step == 0 || step != (size_t)b.row * elem_size(b.dt)) return true;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
    const size_t at = pb >= pa ? (pb - pa) % step : (step - (pa - pb) % step) % step;    // of b's rows behind a's
    return at < wa || at + wb > step;
}
bool same_rows(const Rows &a, const Rows &b) { return a.p == b.p && a.row == b.row && a.dt == b.dt; }

gdn_status check_moe_route(const gdn_moe_params *p)
{
    if (p == nullptr) return fail(GDN_ERR_INVALID_ARG, "moe params is NULL");
    if (p->num_experts < 1 || p->num_experts > GDN_MOE_MAX_EXPERTS)
        return fail(GDN_ERR_INVALID_ARG, "num_experts out of range [1, 256]");
    if (p->top_k < 1 || p->top_k > GDN_MOE_MAX_TOPK || p->top_k > p->num_experts)
        return fail(GDN_ERR_INVALID_ARG, "top_k out of range [1, min(num_experts, 16)]");
    return GDN_OK;
}

gdn_status check_moe_sizes(const gdn_moe_params *p, int M)
{
    const gdn_status st = check_moe_route(p);
    if (st != GDN_OK) return st;
    if (p->ffn_dim < 128 || p->ffn_dim > 8192 || p->ffn_dim % 128)
        return fail(GDN_ERR_INVALID_ARG, "ffn_dim must be a multiple of 128 in [128, 8192]");
    if (M < 0 || M > MAX_T) return fail(GDN_ERR_INVALID_ARG, "M out of range [0, 2^24]");
    return GDN_OK;
}

// chunk_size 0 = library choice: the exact scan for fp32 activations, the
// chunked tensor-core form for bf16 activations.
int resolve_chunk(int chunk_size, gdn_dtype act)
{
    if (chunk_size == 0) return act == GDN_BF16 ? 64 : 1;
    return chunk_size;
}

}  // namespace

namespace gdn {

// Every kernel file keeps its own device error word. gdn_device_error reads and
// clears all of them with one small kernel (an atomic exchange each, so a word
// set while the call runs is either reported now or kept for the next call)
// and one copy of the OR back to the host.
constexpr int N_ERROR_WORDS = 14;
struct ErrorWords {
    unsigned int *p[N_ERROR_WORDS];
};
__device__ unsigned int g_error_any;

__global__ void error_gather_kernel(const ErrorWords w)
{
    if (threadIdx.x != 0) return;
    unsigned int v = 0;
#pragma unroll
    for (int i = 0; i < N_ERROR_WORDS; ++i)
        if (w.p[i]) v |= atomicExch(w.p[i], 0u);
    g_error_any = v;
}

// The words' device addresses, looked up once per device with that device
// current (a host-side symbol is not a device address).
static bool error_words(ErrorWords *out)
{
    constexpr int MAX_DEV = 64;
    static std::mutex mu;
    static ErrorWords cache[MAX_DEV];
    static bool have[MAX_DEV] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= MAX_DEV) return false;
    std::lock_guard<std::mutex> lock(mu);
    if (!have[dev]) {
        void *(*const fns[N_ERROR_WORDS])() = {decode_error_word, chunk_error_word,    multi_error_word,
                                               gemm_error_word,   attn_error_word,     selftest_error_word,
                                               gproj_error_word,  inconv_error_word,   paged_error_word,
                                               paged_q4_error_word, linear_error_word, route_error_word,
                                               moe_error_word,    few_error_word};
        for (int i = 0; i < N_ERROR_WORDS; ++i) {
            cache[dev].p[i] = static_cast<unsigned int *>(fns[i]());
            if (cache[dev].p[i] == nullptr) return false;
        }
        have[dev] = true;
    }
    *out = cache[dev];
    return true;
}

// Lets other translation units of the library set the gdn_last_error() text.
void record_error(const char *msg) { snprintf(g_last_error, sizeof(g_last_error), "%s", msg); }
}  // namespace gdn

extern "C" {

int gdn_abi_version(void) { return GDN_ABI_VERSION; }

const char *gdn_last_error(void) { return g_last_error; }

const char *gdn_status_string(gdn_status s)
{
    switch (s) {
    case GDN_OK: return "GDN_OK";
    case GDN_ERR_INVALID_ARG: return "GDN_ERR_INVALID_ARG";
    case GDN_ERR_UNSUPPORTED: return "GDN_ERR_UNSUPPORTED";
    case GDN_ERR_WORKSPACE: return "GDN_ERR_WORKSPACE";
    case GDN_ERR_CUDA: return "GDN_ERR_CUDA";
    case GDN_ERR_TIMEOUT: return "GDN_ERR_TIMEOUT";
    }
    return "GDN_STATUS_UNKNOWN";
}

gdn_status gdn_conv_step(const float *conv_w, const void *qkv_in, void *qkv_out, void *conv_state, int B,
                         gdn_dtype act, void *stream)
{
    if (!ok_dtype(act)) return fail(GDN_ERR_INVALID_ARG, "unknown activation dtype");
    if (B < 0 || B > MAX_B) return fail(GDN_ERR_INVALID_ARG, "B out of range [0, 65535]");
    if (B == 0) return GDN_OK;
    if (!ok_ptr(conv_w) || !ok_ptr(qkv_in) || !ok_ptr(qkv_out) || !ok_ptr(conv_state))
        return fail(GDN_ERR_INVALID_ARG, "a tensor pointer is NULL or not 16-byte aligned");
    if (qkv_in == qkv_out) return fail(GDN_ERR_INVALID_ARG, "qkv_out may not alias qkv_in");
    cudaError_t e = launch_conv_step(conv_w, qkv_in, qkv_out, conv_state, B, act, (cudaStream_t)stream);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "gdn_conv_step");
}

gdn_status gdn_decode_step(const gdn_params *p, const void *qkv, const void *z, const void *alpha,
                           const void *beta, void *conv_state, float *ssm_state, void *out, int B,
                           gdn_dtype act, gdn_dtype out_dt, void *stream)
{
    if (!ok_dtype(act) || !ok_dtype(out_dt)) return fail(GDN_ERR_INVALID_ARG, "unknown dtype");
    if (B < 0 || B > MAX_B) return fail(GDN_ERR_INVALID_ARG, "B out of range [0, 65535]");
    if (B == 0) return GDN_OK;
    gdn_status st = check_params(p);
    if (st != GDN_OK) return st;
    if (!ok_ptr(qkv) || !ok_ptr(z) || !ok_ptr(alpha) || !ok_ptr(beta) || !ok_ptr(conv_state) ||
        !ok_ptr(ssm_state) || !ok_ptr(out))
        return fail(GDN_ERR_INVALID_ARG, "a tensor pointer is NULL or not 16-byte aligned");
    cudaError_t e = launch_decode_step(p, qkv, z, alpha, beta, conv_state, ssm_state, out, B, act, out_dt,
                                       (cudaStream_t)stream);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "gdn_decode_step");
}

gdn_status gdn_decode_multi(const gdn_params *p, const void *qkv, const void *z, const void *alpha,
                            const void *beta, void *conv_state, float *ssm_state, void *out, int B, int T,
                            gdn_dtype act, gdn_dtype out_dt, void *stream)
{
    if (!ok_dtype(act) || !ok_dtype(out_dt)) return fail(GDN_ERR_INVALID_ARG, "unknown dtype");
    if (B < 0 || B > MAX_B) return fail(GDN_ERR_INVALID_ARG, "B out of range [0, 65535]");
    if (T < 1 || T > GDN_DECODE_MAX_T) return fail(GDN_ERR_INVALID_ARG, "T out of range [1, GDN_DECODE_MAX_T]");
    if (B == 0) return GDN_OK;
    gdn_status st = check_params(p);
    if (st != GDN_OK) return st;
    if (!ok_ptr(qkv) || !ok_ptr(z) || !ok_ptr(alpha) || !ok_ptr(beta) || !ok_ptr(conv_state) ||
        !ok_ptr(ssm_state) || !ok_ptr(out))
        return fail(GDN_ERR_INVALID_ARG, "a tensor pointer is NULL or not 16-byte aligned");
    cudaError_t e = launch_decode_multi(p, qkv, z, alpha, beta, conv_state, ssm_state, out, B, T, act, out_dt,
                                        (cudaStream_t)stream);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "gdn_decode_multi");
}

gdn_status gdn_in_proj(const void *h, const void *w_in, void *qkv, void *z, void *alpha, void *beta, int M,
                       gdn_dtype act, void *stream)
{
    if (!ok_dtype(act)) return fail(GDN_ERR_INVALID_ARG, "unknown activation dtype");
    if (M < 0 || M > (1 << 24)) return fail(GDN_ERR_INVALID_ARG, "M out of range [0, 2^24]");
    if (M == 0) return GDN_OK;
    if (!ok_ptr(h) || !ok_ptr(w_in) || !ok_ptr(qkv) || !ok_ptr(z) || !ok_ptr(alpha) || !ok_ptr(beta))
        return fail(GDN_ERR_INVALID_ARG, "a tensor pointer is NULL or not 16-byte aligned");
    cudaError_t e = launch_in_proj(h, w_in, qkv, z, alpha, beta, M, act, (cudaStream_t)stream);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "gdn_in_proj");
}

gdn_status gdn_out_proj(const void *x, const void *w, void *y, int M, gdn_dtype out_dt, void *stream)
{
    if (!ok_dtype(out_dt)) return fail(GDN_ERR_INVALID_ARG, "unknown output dtype");
    if (M < 0 || M > (1 << 24)) return fail(GDN_ERR_INVALID_ARG, "M out of range [0, 2^24]");
    if (M == 0) return GDN_OK;
    if (!ok_ptr(x) || !ok_ptr(w) || !ok_ptr(y))
        return fail(GDN_ERR_INVALID_ARG, "a tensor pointer is NULL or not 16-byte aligned");
    cudaError_t e = launch_out_proj(x, w, y, M, out_dt, (cudaStream_t)stream);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "gdn_out_proj");
}

gdn_status gdn_gated_out_proj(const float *norm_w, float norm_eps, const void *y, const void *z, const void *w,
                              void *out, int M, gdn_dtype act, gdn_dtype out_dt, void *stream)
{
    if (!ok_dtype(act) || !ok_dtype(out_dt)) return fail(GDN_ERR_INVALID_ARG, "unknown activation or output dtype");
    if (M < 0 || M > (1 << 24)) return fail(GDN_ERR_INVALID_ARG, "M out of range [0, 2^24]");
    if (M == 0) return GDN_OK;
    if (!ok_ptr(norm_w) || !ok_ptr(y) || !ok_ptr(z) || !ok_ptr(w) || !ok_ptr(out))
        return fail(GDN_ERR_INVALID_ARG, "a tensor pointer is NULL or not 16-byte aligned");
    if (!(norm_eps >= 0.0f)) return fail(GDN_ERR_INVALID_ARG, "norm_eps must be >= 0");
    cudaError_t e = launch_gated_out_proj(norm_w, norm_eps, y, z, w, out, M, act, out_dt, (cudaStream_t)stream);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "gdn_gated_out_proj");
}

size_t gdn_attn_decode_workspace_size(int B, int Lmax)
{
    if (B < 1 || B > MAX_B || Lmax < 1 || (long long)B * GDN_ATTN_KV_HEADS * Lmax > (1ll << 30)) return 0;
    return attn_workspace_bytes(B, Lmax);
}

gdn_status gdn_attn_decode(const void *q, const void *k_cache, const void *v_cache, const int32_t *ctx_len,
                           const void *z, void *out, int B, int Lmax, void *workspace, size_t workspace_bytes,
                           gdn_dtype out_dt, void *stream)
{
    if (!ok_dtype(out_dt)) return fail(GDN_ERR_INVALID_ARG, "unknown output dtype");
    if (B < 0 || B > MAX_B) return fail(GDN_ERR_INVALID_ARG, "B out of range [0, 65535]");
    if (B == 0) return GDN_OK;
    if (Lmax < 1 || (long long)B * GDN_ATTN_KV_HEADS * Lmax > (1ll << 30))
        return fail(GDN_ERR_INVALID_ARG, "Lmax out of range: need 1 <= Lmax and B * 2 * Lmax <= 2^30");
    if (!ok_ptr(q) || !ok_ptr(k_cache) || !ok_ptr(v_cache) || !ok_ptr(z) || !ok_ptr(out))
        return fail(GDN_ERR_INVALID_ARG, "a tensor pointer is NULL or not 16-byte aligned");
    if (ctx_len == nullptr || (reinterpret_cast<uintptr_t>(ctx_len) & 3u) != 0)
        return fail(GDN_ERR_INVALID_ARG, "ctx_len is NULL or not 4-byte aligned");
    if (!ok_ptr(workspace)) return fail(GDN_ERR_WORKSPACE, "workspace is NULL or not 16-byte aligned");
    if (workspace_bytes < attn_workspace_bytes(B, Lmax))
        return fail(GDN_ERR_WORKSPACE, "workspace smaller than gdn_attn_decode_workspace_size(B, Lmax)");
    cudaError_t e = launch_attn_decode(q, k_cache, v_cache, ctx_len, z, out, B, Lmax, workspace, out_dt,
                                       (cudaStream_t)stream);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "gdn_attn_decode");
}

gdn_status gdn_attn_qk_norm_rope(const gdn_attn_params *p, const void *q, long long q_row_stride,
                                 long long q_head_stride, const void *k, long long k_row_stride,
                                 long long k_head_stride, const int32_t *positions, int M, void *q_out, void *k_out,
                                 gdn_dtype act, gdn_dtype out_dt, void *stream)
{
    if (!ok_dtype(act) || !ok_dtype(out_dt)) return fail(GDN_ERR_INVALID_ARG, "unknown activation or output dtype");
    if (M < 0 || M > MAX_T) return fail(GDN_ERR_INVALID_ARG, "M out of range [0, 2^24]");
    gdn_status st = check_attn_params(p);
    if (st != GDN_OK || M == 0) return st;
    const Heads hq = {q, q_row_stride, q_head_stride, GDN_ATTN_Q_HEADS, act};
    const Heads hk = {k, k_row_stride, k_head_stride, GDN_ATTN_KV_HEADS, act};
    if ((st = check_heads(hq)) != GDN_OK) return st;
    if (k != nullptr && (st = check_heads(hk)) != GDN_OK) return st;
    if (!ok_ptr(q_out) || (k != nullptr) != (k_out != nullptr) || !ok_opt_ptr(k_out))
        return fail(GDN_ERR_INVALID_ARG, "an output is NULL or not 16-byte aligned, or only one of k and k_out is given");
    if (p->rope != nullptr && (positions == nullptr || !aligned4(positions)))
        return fail(GDN_ERR_INVALID_ARG, "positions is NULL or not 4-byte aligned");
    const size_t es = out_dt == GDN_F32 ? 4 : 2, qo = (size_t)M * GDN_ATTN_Q_HEADS * GDN_ATTN_HEAD_DIM * es,
                 ko = (size_t)M * GDN_ATTN_KV_HEADS * GDN_ATTN_HEAD_DIM * es;
    const bool q_same = q_out == q && hq.dense() && act == out_dt, k_same = k_out == k && hk.dense() && act == out_dt;
    if ((!q_same && overlap(q_out, qo, q, hq.bytes(M))) ||
        (k != nullptr && ((!k_same && overlap(k_out, ko, k, hk.bytes(M))) || overlap(q_out, qo, k, hk.bytes(M)) ||
                          overlap(k_out, ko, q, hq.bytes(M)) || overlap(q_out, qo, k_out, ko))))
        return fail(GDN_ERR_INVALID_ARG, "an output overlaps an input or the other output");
    cudaError_t e = launch_qk_norm_rope(p, q, q_row_stride, q_head_stride, k, k_row_stride, k_head_stride, positions,
                                        M, q_out, k_out, act, out_dt, (cudaStream_t)stream);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "gdn_attn_qk_norm_rope");
}

gdn_status gdn_kv_append(const gdn_attn_params *p, const gdn_paged_batch *batch, const gdn_kv_cache *cache,
                         const void *k, long long k_row_stride, long long k_head_stride, const void *v,
                         long long v_row_stride, long long v_head_stride, const void *q, long long q_row_stride,
                         long long q_head_stride, void *q_out, const int32_t *positions, gdn_dtype act,
                         void *stream)
{
    if (!ok_dtype(act)) return fail(GDN_ERR_INVALID_ARG, "unknown activation dtype");
    gdn_status st = check_attn_params(p);
    if (st == GDN_OK) st = check_batch(batch, cache);
    if (st != GDN_OK || batch->B == 0 || batch->M == 0) return st;
    const int M = batch->M;
    const Heads hk = {k, k_row_stride, k_head_stride, GDN_ATTN_KV_HEADS, act};
    const Heads hv = {v, v_row_stride, v_head_stride, GDN_ATTN_KV_HEADS, act};
    const Heads hq = {q, q_row_stride, q_head_stride, GDN_ATTN_Q_HEADS, act};
    if ((st = check_heads(hk)) != GDN_OK || (st = check_heads(hv)) != GDN_OK) return st;
    if (q != nullptr && (st = check_heads(hq)) != GDN_OK) return st;
    if ((q != nullptr) != (q_out != nullptr) || !ok_opt_ptr(q_out))
        return fail(GDN_ERR_INVALID_ARG, "q_out is not 16-byte aligned, or only one of q and q_out is given");
    if (!aligned4(positions)) return fail(GDN_ERR_INVALID_ARG, "positions is not 4-byte aligned");
    const size_t cb = kv_cache_bytes(cache), qo = (size_t)M * GDN_ATTN_Q_HEADS * GDN_ATTN_HEAD_DIM * 2;
    const Heads ins[3] = {hk, hv, hq};
    for (const Heads &t : ins) {
        if (t.p == nullptr) continue;
        const bool same = q_out != nullptr && t.p == q && q_out == q && hq.dense() && act == GDN_BF16;
        if (overlap(cache->k, cb, t.p, t.bytes(M)) || (cache->v && overlap(cache->v, cb, t.p, t.bytes(M))) ||
            (q_out != nullptr && !same && overlap(q_out, qo, t.p, t.bytes(M))))
            return fail(GDN_ERR_INVALID_ARG, "the cache or q_out overlaps an input");
    }
    if (q_out != nullptr && (overlap(cache->k, cb, q_out, qo) || (cache->v && overlap(cache->v, cb, q_out, qo))))
        return fail(GDN_ERR_INVALID_ARG, "the cache overlaps q_out");
    cudaError_t e = launch_kv_append(p, batch, cache, k, k_row_stride, k_head_stride, v, v_row_stride, v_head_stride,
                                     q, q_row_stride, q_head_stride, q_out, positions, act, (cudaStream_t)stream);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "gdn_kv_append");
}

gdn_status gdn_kv_gather(const gdn_paged_batch *batch, const gdn_kv_cache *cache, void *k_out, void *v_out,
                         gdn_dtype out_dt, void *stream)
{
    if (!ok_dtype(out_dt)) return fail(GDN_ERR_INVALID_ARG, "unknown output dtype");
    gdn_status st = check_batch(batch, cache);
    if (st != GDN_OK || batch->B == 0 || batch->M == 0) return st;
    if (!ok_opt_ptr(k_out) || !ok_opt_ptr(v_out)) return fail(GDN_ERR_INVALID_ARG, "an output is not 16-byte aligned");
    if (k_out == nullptr && v_out == nullptr) return GDN_OK;
    const size_t n = (size_t)batch->M * GDN_ATTN_KV_HEADS * GDN_ATTN_HEAD_DIM * (out_dt == GDN_F32 ? 4 : 2);
    const size_t cb = kv_cache_bytes(cache);
    void *const outs[2] = {k_out, v_out};
    for (void *o : outs)
        if (o && (overlap(o, n, cache->k, cb) || (cache->v && overlap(o, n, cache->v, cb))))
            return fail(GDN_ERR_INVALID_ARG, "an output overlaps the cache");
    if (k_out && v_out && overlap(k_out, n, v_out, n)) return fail(GDN_ERR_INVALID_ARG, "k_out and v_out overlap");
    cudaError_t e = launch_kv_gather(batch, cache, k_out, v_out, out_dt, (cudaStream_t)stream);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "gdn_kv_gather");
}

size_t gdn_attn_paged_workspace_size(const gdn_paged_batch *batch, const gdn_kv_cache *cache)
{
    if (check_batch_sizes(batch, cache) != GDN_OK) return 0;
    return paged_workspace_bytes(batch, cache);
}

gdn_status gdn_attn_paged(const gdn_paged_batch *batch, const gdn_kv_cache *cache, const void *q, const void *gate,
                          long long gate_row_stride, long long gate_head_stride, void *out, void *workspace,
                          size_t workspace_bytes, gdn_dtype out_dt, void *stream)
{
    if (!ok_dtype(out_dt)) return fail(GDN_ERR_INVALID_ARG, "unknown output dtype");
    gdn_status st = check_batch(batch, cache);
    if (st != GDN_OK || batch->B == 0 || batch->M == 0) return st;
    if (!ok_ptr(q) || !ok_ptr(out)) return fail(GDN_ERR_INVALID_ARG, "a tensor pointer is NULL or not 16-byte aligned");
    const Heads hg = {gate, gate_row_stride, gate_head_stride, GDN_ATTN_Q_HEADS, GDN_BF16};
    if (gate != nullptr && (st = check_heads(hg)) != GDN_OK) return st;
    const size_t n = (size_t)batch->M * GDN_ATTN_Q_HEADS * GDN_ATTN_HEAD_DIM, no = n * (out_dt == GDN_F32 ? 4 : 2);
    const size_t cb = kv_cache_bytes(cache);
    if (overlap(out, no, q, n * 2) || (gate && overlap(out, no, gate, hg.bytes(batch->M))) ||
        overlap(out, no, cache->k, cb) || (cache->v && overlap(out, no, cache->v, cb)))
        return fail(GDN_ERR_INVALID_ARG, "out overlaps an input");
    if (!ok_ptr(workspace)) return fail(GDN_ERR_WORKSPACE, "workspace is NULL or not 16-byte aligned");
    if (workspace_bytes < paged_workspace_bytes(batch, cache))
        return fail(GDN_ERR_WORKSPACE, "workspace smaller than gdn_attn_paged_workspace_size(batch, cache)");
    cudaError_t e = launch_attn_paged(batch, cache, q, gate, gate_row_stride, gate_head_stride, out, workspace, out_dt,
                                      (cudaStream_t)stream);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "gdn_attn_paged");
}

size_t gdn_prefill_workspace_size(int N, int T_total, gdn_dtype act, int chunk_size)
{
    if (N < 0 || N > MAX_N || T_total < 0 || T_total > MAX_T || !ok_dtype(act)) return 0;
    const int ch = resolve_chunk(chunk_size, act);
    size_t body = 0;
    if (ch == 1) body = scan_workspace_bytes(T_total);
    else if (ch == 64 && act == GDN_BF16) body = chunk_workspace_bytes(N, T_total);
    else return 0;
    return WS_HEADER + ((body + 255) & ~(size_t)255);
}

gdn_status gdn_prefill(const gdn_params *p, const void *qkv, const void *z, const void *alpha, const void *beta,
                       const int32_t *cu_seqlens, int N, int T_total, const void *conv_state_in,
                       void *conv_state_out, const float *ssm_state_in, float *ssm_state_out, void *out,
                       gdn_dtype act, gdn_dtype out_dt, int chunk_size, void *workspace, size_t ws_bytes,
                       void *stream)
{
    if (!ok_dtype(act) || !ok_dtype(out_dt)) return fail(GDN_ERR_INVALID_ARG, "unknown dtype");
    if (N < 0 || N > MAX_N) return fail(GDN_ERR_INVALID_ARG, "N out of range [0, 65535]");
    if (T_total < 0 || T_total > MAX_T) return fail(GDN_ERR_INVALID_ARG, "T_total out of range [0, 2^24]");
    if (N == 0) {
        if (T_total != 0) return fail(GDN_ERR_INVALID_ARG, "T_total > 0 with no sequences");
        return GDN_OK;
    }
    const int ch = resolve_chunk(chunk_size, act);
    if (ch != 1 && ch != 64) return fail(GDN_ERR_UNSUPPORTED, "chunk_size must be 0, 1 or 64");
    if (ch == 64 && act != GDN_BF16)
        return fail(GDN_ERR_UNSUPPORTED, "the chunked tensor-core form needs bf16 activations");
    gdn_status st = check_params(p);
    if (st != GDN_OK) return st;
    if (!ok_ptr(cu_seqlens) || (T_total > 0 && (!ok_ptr(qkv) || !ok_ptr(z) || !ok_ptr(alpha) ||
                                                !ok_ptr(beta) || !ok_ptr(out))))
        return fail(GDN_ERR_INVALID_ARG, "a tensor pointer is NULL or not 16-byte aligned");
    if (!ok_opt_ptr(conv_state_in) || !ok_opt_ptr(conv_state_out) || !ok_opt_ptr(ssm_state_in) ||
        !ok_opt_ptr(ssm_state_out))
        return fail(GDN_ERR_INVALID_ARG, "a state pointer is not 16-byte aligned");
    // The exact scan needs its whole workspace. The chunked form runs in windows
    // of the packed tokens sized to the workspace it is given, so any workspace
    // that holds one 64-token window will do.
    const size_t need = ch == 1 ? gdn_prefill_workspace_size(N, T_total, act, ch)
                                : WS_HEADER + ((chunk_min_workspace_bytes(N) + 255) & ~(size_t)255);
    if (workspace == nullptr || ws_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u)) {
        snprintf(g_last_error, sizeof(g_last_error),
                 "workspace missing, misaligned (256 B) or too small: %zu bytes given, %zu needed", ws_bytes, need);
        return GDN_ERR_WORKSPACE;
    }
    void *body = static_cast<char *>(workspace) + WS_HEADER;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (ch == 1)
        e = launch_prefill_scan(p, qkv, z, alpha, beta, cu_seqlens, N, T_total, conv_state_in, conv_state_out,
                                ssm_state_in, ssm_state_out, out, act, out_dt, body, s);
    else
        e = launch_prefill_chunked(p, qkv, z, alpha, beta, cu_seqlens, N, T_total, conv_state_in, conv_state_out,
                                   ssm_state_in, ssm_state_out, out, out_dt, body, ws_bytes - WS_HEADER, s, nullptr);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "gdn_prefill");
}

gdn_status gdn_in_proj_conv(const gdn_params *p, const void *h, const void *w_in, const int32_t *cu_seqlens, int N,
                            int M, const void *conv_state_in, void *conv_state_out, void *xhat, void *z,
                            void *alpha, void *beta, void *stream)
{
    if (N < 0 || N > MAX_N) return fail(GDN_ERR_INVALID_ARG, "N out of range [0, 65535]");
    if (M < 0 || M > MAX_T) return fail(GDN_ERR_INVALID_ARG, "M out of range [0, 2^24]");
    if (N == 0) {
        if (M != 0) return fail(GDN_ERR_INVALID_ARG, "M > 0 with no sequences");
        return GDN_OK;
    }
    if (p == nullptr || !ok_ptr(p->conv_w) || !(p->l2_eps >= 0.0f))
        return fail(GDN_ERR_INVALID_ARG, "params NULL, conv_w NULL or misaligned, or l2_eps < 0");
    if (!ok_ptr(cu_seqlens) || (M > 0 && (!ok_ptr(h) || !ok_ptr(w_in) || !ok_ptr(xhat) || !ok_ptr(z) ||
                                          !ok_ptr(alpha) || !ok_ptr(beta))))
        return fail(GDN_ERR_INVALID_ARG, "a tensor pointer is NULL or not 16-byte aligned");
    if (!ok_opt_ptr(conv_state_in) || !ok_opt_ptr(conv_state_out))
        return fail(GDN_ERR_INVALID_ARG, "a state pointer is not 16-byte aligned");
    const size_t cs_bytes = (size_t)N * (GDN_CONV_K - 1) * GDN_CONV_CHANNELS * 2;
    if (conv_state_in && conv_state_out) {
        const char *i0 = static_cast<const char *>(conv_state_in), *o0 = static_cast<const char *>(conv_state_out);
        if (i0 < o0 + cs_bytes && o0 < i0 + cs_bytes)
            return fail(GDN_ERR_INVALID_ARG, "conv_state_in and conv_state_out overlap");
    }
    cudaError_t e = launch_in_proj_conv(p->conv_w, p->l2_eps, h, w_in, cu_seqlens, N, M, conv_state_in,
                                        conv_state_out, xhat, z, alpha, beta, (cudaStream_t)stream);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "gdn_in_proj_conv");
}

gdn_status gdn_prefill_xhat(const gdn_params *p, const void *xhat, const void *z, const void *alpha,
                            const void *beta, const int32_t *cu_seqlens, int N, int T_total,
                            const float *ssm_state_in, float *ssm_state_out, void *out, gdn_dtype out_dt,
                            void *workspace, size_t ws_bytes, void *stream)
{
    if (!ok_dtype(out_dt)) return fail(GDN_ERR_INVALID_ARG, "unknown dtype");
    if (N < 0 || N > MAX_N) return fail(GDN_ERR_INVALID_ARG, "N out of range [0, 65535]");
    if (T_total < 0 || T_total > MAX_T) return fail(GDN_ERR_INVALID_ARG, "T_total out of range [0, 2^24]");
    if (N == 0) {
        if (T_total != 0) return fail(GDN_ERR_INVALID_ARG, "T_total > 0 with no sequences");
        return GDN_OK;
    }
    gdn_status st = check_params(p);
    if (st != GDN_OK) return st;
    if (!ok_ptr(cu_seqlens) || (T_total > 0 && (!ok_ptr(xhat) || !ok_ptr(z) || !ok_ptr(alpha) || !ok_ptr(beta) ||
                                                !ok_ptr(out))))
        return fail(GDN_ERR_INVALID_ARG, "a tensor pointer is NULL or not 16-byte aligned");
    if (!ok_opt_ptr(ssm_state_in) || !ok_opt_ptr(ssm_state_out))
        return fail(GDN_ERR_INVALID_ARG, "a state pointer is not 16-byte aligned");
    const size_t need = WS_HEADER + ((chunk_min_workspace_bytes(N) + 255) & ~(size_t)255);
    if (workspace == nullptr || ws_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u)) {
        snprintf(g_last_error, sizeof(g_last_error),
                 "workspace missing, misaligned (256 B) or too small: %zu bytes given, %zu needed", ws_bytes, need);
        return GDN_ERR_WORKSPACE;
    }
    void *body = static_cast<char *>(workspace) + WS_HEADER;
    cudaError_t e = launch_prefill_chunked(p, nullptr, z, alpha, beta, cu_seqlens, N, T_total, nullptr, nullptr,
                                           ssm_state_in, ssm_state_out, out, out_dt, body, ws_bytes - WS_HEADER,
                                           (cudaStream_t)stream, xhat);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "gdn_prefill_xhat");
}

gdn_status gdn_add_norm(const gdn_norm_params *p, const void *x, long long x_row_stride, const void *delta,
                        long long delta_row_stride, const void *gate, long long gate_row_stride, void *x_out,
                        long long x_out_row_stride, void *h, long long h_row_stride, int M, gdn_dtype stream_dt,
                        gdn_dtype act, void *stream)
{
    if (!ok_dtype(stream_dt) || !ok_dtype(act)) return fail(GDN_ERR_INVALID_ARG, "unknown dtype");
    if (p == nullptr) return fail(GDN_ERR_INVALID_ARG, "norm params is NULL");
    if (M < 0 || M > MAX_T) return fail(GDN_ERR_INVALID_ARG, "M out of range [0, 2^24]");
    if (!ok_opt_ptr(p->norm_w) || !ok_opt_ptr(p->post_w) || (h != nullptr && p->norm_w == nullptr))
        return fail(GDN_ERR_INVALID_ARG, "a norm weight is not 16-byte aligned, or norm_w is NULL with an output h");
    if (!(p->norm_eps >= 0.0f)) return fail(GDN_ERR_INVALID_ARG, "norm_eps must be >= 0");
    if (M == 0) return GDN_OK;
    if (delta == nullptr && gate != nullptr) return fail(GDN_ERR_INVALID_ARG, "gate without delta");
    if (x_out == nullptr && h == nullptr) return fail(GDN_ERR_INVALID_ARG, "no output");
    const Rows rx = {x, x_row_stride, GDN_HIDDEN, stream_dt}, rd = {delta, delta_row_stride, GDN_HIDDEN, act},
               rg = {gate, gate_row_stride, GDN_HIDDEN, act}, ro = {x_out, x_out_row_stride, GDN_HIDDEN, stream_dt},
               rh = {h, h_row_stride, GDN_HIDDEN, act};
    if (!rx.ok() || (delta && !rd.ok()) || (gate && !rg.ok(true)) || (x_out && !ro.ok()) || (h && !rh.ok()))
        return fail(GDN_ERR_INVALID_ARG,
                    "a tensor is NULL or not 16-byte aligned, or a row stride is below 2048 or not a multiple of 16 bytes");
    if ((overlap(ro, rx, M) && !same_rows(ro, rx)) || overlap(ro, rd, M) || overlap(ro, rg, M) || overlap(ro, rh, M) ||
        (overlap(rh, rd, M) && !same_rows(rh, rd)) || overlap(rh, rx, M) || overlap(rh, rg, M))
        return fail(GDN_ERR_INVALID_ARG, "an output overlaps another tensor");
    const float *const norm_weights[] = {p->norm_w, p->post_w};
    for (const float *w : norm_weights)
        if (w && ((x_out && overlap(x_out, ro.bytes(M), w, GDN_HIDDEN * 4)) || (h && overlap(h, rh.bytes(M), w, GDN_HIDDEN * 4))))
            return fail(GDN_ERR_INVALID_ARG, "an output overlaps a norm weight");
    cudaError_t e = launch_add_norm(p, x, x_row_stride, delta, delta_row_stride, gate, gate_row_stride, x_out,
                                    x_out_row_stride, h, h_row_stride, M, stream_dt, act, (cudaStream_t)stream);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "gdn_add_norm");
}

gdn_status gdn_linear(const void *x, long long x_row_stride, const void *w, const float *bias, const void *residual,
                      long long residual_row_stride, void *y, long long y_row_stride, int M, int N, int K,
                      gdn_activation activation, gdn_dtype out_dt, void *stream)
{
    if (!ok_dtype(out_dt)) return fail(GDN_ERR_INVALID_ARG, "unknown output dtype");
    if (activation != GDN_ACT_NONE && activation != GDN_ACT_SILU && activation != GDN_ACT_GELU &&
        activation != GDN_ACT_SIGMOID)
        return fail(GDN_ERR_INVALID_ARG, "unknown activation");
    if (M < 0 || M > MAX_T) return fail(GDN_ERR_INVALID_ARG, "M out of range [0, 2^24]");
    if (N < 8 || N > (1 << 20) || N % 8 || K < 8 || K > (1 << 20) || K % 8)
        return fail(GDN_ERR_INVALID_ARG, "N and K must be multiples of 8 in [8, 2^20]");
    if (M == 0) return GDN_OK;
    const Rows rx = {x, x_row_stride, K, GDN_BF16}, rw = {w, K, K, GDN_BF16},
               rr = {residual, residual_row_stride, N, out_dt}, ry = {y, y_row_stride, N, out_dt};
    if (!rx.ok() || !rw.ok() || !ok_opt_ptr(bias) || (residual && !rr.ok()) || !ry.ok())
        return fail(GDN_ERR_INVALID_ARG,
                    "a tensor is NULL or not 16-byte aligned, or a row stride is below the row or not a multiple of 16 bytes");
    if (overlap(ry, rx, M) || overlap(y, ry.bytes(M), w, rw.bytes(N)) || (overlap(ry, rr, M) && !same_rows(ry, rr)) ||
        (bias && overlap(y, ry.bytes(M), bias, (size_t)N * 4)))
        return fail(GDN_ERR_INVALID_ARG, "y overlaps an input");
    cudaError_t e = launch_linear(x, x_row_stride, w, bias, residual, residual_row_stride, y, y_row_stride, M, N, K,
                                  activation, out_dt, (cudaStream_t)stream);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "gdn_linear");
}

gdn_status gdn_moe_route(const gdn_moe_params *p, const void *x, long long x_row_stride, int M, int32_t *ids,
                         float *weights, void *stream)
{
    gdn_status st = check_moe_route(p);
    if (st != GDN_OK) return st;
    if (M < 0 || M > MAX_T) return fail(GDN_ERR_INVALID_ARG, "M out of range [0, 2^24]");
    if (M == 0) return GDN_OK;
    const Rows rx = {x, x_row_stride, GDN_HIDDEN, GDN_BF16};
    if (!rx.ok() || !ok_ptr(p->router) || !ok_ptr(ids) || !ok_ptr(weights))
        return fail(GDN_ERR_INVALID_ARG, "a tensor is NULL or not 16-byte aligned, or the row stride is below 2048 or not a multiple of 8");
    const size_t n = (size_t)M * p->top_k * 4, nr = (size_t)p->num_experts * GDN_HIDDEN * 2;
    if (overlap(ids, n, weights, n) || overlap(ids, n, x, rx.bytes(M)) || overlap(weights, n, x, rx.bytes(M)) ||
        overlap(ids, n, p->router, nr) || overlap(weights, n, p->router, nr))
        return fail(GDN_ERR_INVALID_ARG, "an output overlaps another tensor");
    cudaError_t e = launch_route_only(p, x, x_row_stride, M, ids, weights, (cudaStream_t)stream);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "gdn_moe_route");
}

size_t gdn_moe_workspace_size(const gdn_moe_params *p, int M)
{
    if (check_moe_sizes(p, M) != GDN_OK) return 0;
    return moe_workspace_bytes(p, M);
}

static gdn_status moe_call(const gdn_moe_params *p, const void *x, long long x_row_stride, const void *residual, void *out,
                           int M, const int32_t *ids, const float *weights, void *workspace, size_t workspace_bytes,
                           gdn_dtype out_dt, bool lose_route, void *stream)
{
    if (!ok_dtype(out_dt)) return fail(GDN_ERR_INVALID_ARG, "unknown output dtype");
    gdn_status st = check_moe_sizes(p, M);
    if (st != GDN_OK || M == 0) return st;
    if (lose_route && M <= 4) return fail(GDN_ERR_INVALID_ARG, "M must be above 4");
    if ((ids == nullptr) != (weights == nullptr)) return fail(GDN_ERR_INVALID_ARG, "ids and weights go together");
    if ((p->sh_gate == nullptr) != (p->sh_up == nullptr) || (p->sh_gate == nullptr) != (p->sh_down == nullptr) ||
        (p->sh_gate == nullptr && p->sh_router != nullptr))
        return fail(GDN_ERR_INVALID_ARG, "the shared expert's tensors go together");
    const Rows rx = {x, x_row_stride, GDN_HIDDEN, GDN_BF16};
    if (!rx.ok() || !ok_opt_ptr(residual) || !ok_ptr(out) || !ok_ptr(p->gate) || !ok_ptr(p->up) || !ok_ptr(p->down) ||
        !ok_opt_ptr(p->sh_gate) || !ok_opt_ptr(p->sh_up) || !ok_opt_ptr(p->sh_down) || !ok_opt_ptr(p->sh_router) ||
        !ok_opt_ptr(ids) || !ok_opt_ptr(weights) || (ids == nullptr && !ok_ptr(p->router)) || !ok_opt_ptr(p->router))
        return fail(GDN_ERR_INVALID_ARG, "a tensor is NULL or not 16-byte aligned, or the row stride is below 2048 or not a multiple of 8");
    const size_t no = (size_t)M * GDN_HIDDEN * elem_size(out_dt), nx = rx.bytes(M), np = (size_t)M * p->top_k * 4;
    const size_t nf = (size_t)p->ffn_dim * GDN_HIDDEN * 2, ne = (size_t)p->num_experts * nf;
    const size_t need = moe_call_bytes(p, M);
    struct { const void *q; size_t n; } in[] = {
        {x, nx}, {p->gate, ne}, {p->up, ne}, {p->down, ne}, {p->sh_gate, p->sh_gate ? nf : 0}, {p->sh_up, p->sh_up ? nf : 0},
        {p->sh_down, p->sh_down ? nf : 0}, {p->sh_router, p->sh_router ? (size_t)GDN_HIDDEN * 2 : 0},
        {p->router, p->router ? (size_t)p->num_experts * GDN_HIDDEN * 2 : 0}, {ids, ids ? np : 0}, {weights, ids ? np : 0},
        {residual, residual && residual != out ? no : 0}};
    for (const auto &t : in)
        if (overlap(out, no, t.q, t.n)) return fail(GDN_ERR_INVALID_ARG, "out overlaps an input");
    if (workspace == nullptr || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u)) {
        snprintf(g_last_error, sizeof(g_last_error),
                 "workspace missing, misaligned (256 B) or too small: %zu bytes given, %zu needed", workspace_bytes, need);
        return GDN_ERR_WORKSPACE;
    }
    for (const auto &t : in)
        if (overlap(workspace, need, t.q, t.n)) return fail(GDN_ERR_INVALID_ARG, "the workspace overlaps an input");
    if (overlap(workspace, need, out, no)) return fail(GDN_ERR_INVALID_ARG, "the workspace overlaps out");
    cudaError_t e = launch_moe(p, x, x_row_stride, residual, out, M, ids, weights, workspace, out_dt, lose_route,
                               (cudaStream_t)stream);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "gdn_moe");
}

gdn_status gdn_moe(const gdn_moe_params *p, const void *x, long long x_row_stride, const void *residual, void *out,
                   int M, const int32_t *ids, const float *weights, void *workspace, size_t workspace_bytes,
                   gdn_dtype out_dt, void *stream)
{
    return moe_call(p, x, x_row_stride, residual, out, M, ids, weights, workspace, workspace_bytes, out_dt, false, stream);
}

gdn_status gdn_selftest_moe_lost_route(const gdn_moe_params *p, const void *x, long long x_row_stride,
                                       const void *residual, void *out, int M, void *workspace, size_t workspace_bytes,
                                       gdn_dtype out_dt, void *stream)
{
    return moe_call(p, x, x_row_stride, residual, out, M, nullptr, nullptr, workspace, workspace_bytes, out_dt, true, stream);
}

gdn_status gdn_device_error(void *stream)
{
    cudaStream_t s = (cudaStream_t)stream;
    ErrorWords w;
    if (!error_words(&w)) return cuda_fail(cudaGetLastError(), "gdn_device_error: error word lookup");
    unsigned int any = 0;
    error_gather_kernel<<<1, 32, 0, s>>>(w);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) e = cudaMemcpyFromSymbolAsync(&any, g_error_any, sizeof(unsigned int), 0,
                                                        cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return cuda_fail(e, "gdn_device_error");
    return any == 0 ? GDN_OK : GDN_ERR_TIMEOUT;
}

gdn_status gdn_get_device_error(void *workspace, void *stream)
{
    (void)workspace;
    return gdn_device_error(stream);
}

gdn_status gdn_selftest_wait_timeout(void *stream)
{
    cudaError_t e = launch_wait_timeout((cudaStream_t)stream);
    return e == cudaSuccess ? GDN_OK : cuda_fail(e, "gdn_selftest_wait_timeout");
}

}  // extern "C"
