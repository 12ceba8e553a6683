// C ABI of the key/value cache calls (include/nvfp4.h): argument validation on the host, then kernel
// launches on the caller's stream. Every check runs before anything is enqueued.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/nvfp4.h"
#include "kv_cache.h"

namespace {

constexpr int64_t kInt32 = (int64_t)1 << 31;
constexpr int64_t kMaxSpan = (int64_t)1 << 56;

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool span_ok(int64_t n, int64_t stride) {
    return stride <= kMaxSpan && (n <= 1 || stride <= kMaxSpan / n);
}
nvfp4_status hip_status(hipError_t e) { return e == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP; }

int elem_size(int dtype) {
    if (dtype == NVFP4_DTYPE_F32) return 4;
    if (dtype == NVFP4_DTYPE_BF16) return 2;
    return 0;
}

bool layout_ok(int64_t heads, int64_t dim, int64_t page) {
    return heads >= 1 && heads <= 65535 && (dim == 64 || dim == 128 || dim == 256) && page >= 16 &&
           page % 16 == 0 && nvfp4::kv_record_bytes(heads, dim, page) < kInt32;
}

// What every call needs of a cache. `tokens`: a token call (S_k, S_v), else a page call (refs).
nvfp4_status check_cache(const nvfp4_kv_cache* c, bool tokens) {
    if (c == nullptr) return NVFP4_ERR_NULL;
    if (!layout_ok(c->heads, c->head_dim, c->page_size)) return NVFP4_ERR_SHAPE;
    const int64_t rec = nvfp4::kv_record_bytes(c->heads, c->head_dim, c->page_size);
    if (c->layers < 1 || c->layers > 65535 || c->num_pages < 0 || c->num_pages >= kInt32 - 4096 ||
        c->max_slots < 0 || c->max_slots > 65536 || c->max_pages < 0 ||
        (int64_t)c->max_pages * c->page_size > kInt32 - 65536 || c->max_slots * c->max_pages >= kInt32)
        return NVFP4_ERR_SHAPE;
    if (c->page_stride < rec || !span_ok(c->num_pages, c->page_stride)) return NVFP4_ERR_SHAPE;
    if (c->layers > 1 && (c->layer_stride < c->num_pages * c->page_stride ||
                          !span_ok(c->layers, c->layer_stride)))
        return NVFP4_ERR_SHAPE;
    if ((c->num_pages > 0 && c->pages == nullptr) || c->lens == nullptr ||
        (c->max_pages > 0 && c->table == nullptr))
        return NVFP4_ERR_NULL;
    if (tokens ? (c->S_k == nullptr || c->S_v == nullptr) : (c->num_pages > 0 && c->refs == nullptr))
        return NVFP4_ERR_NULL;
    if (!aligned(c->pages, 16) || c->page_stride % 16 != 0 ||
        (c->layers > 1 && c->layer_stride % 16 != 0) || !aligned(c->table, 4) ||
        !aligned(c->lens, 4) || !aligned(c->refs, 4) || !aligned(c->S_k, 4) || !aligned(c->S_v, 4))
        return NVFP4_ERR_ALIGN;
    return NVFP4_OK;
}

nvfp4::KvView view_of(const nvfp4_kv_cache* c, int64_t layer) {
    nvfp4::KvView v;
    v.pages = c->pages + (c->layers > 1 ? layer * c->layer_stride : 0);
    v.page_stride = c->page_stride;
    v.num_pages = (int32_t)c->num_pages;
    v.heads = c->heads;
    v.dim = c->head_dim;
    v.page = c->page_size;
    v.max_slots = (int32_t)c->max_slots;
    v.max_pages = c->max_pages;
    v.table = c->table;
    v.lens = c->lens;
    v.S_k = c->S_k + layer * c->heads;
    v.S_v = c->S_v + layer * c->heads;
    return v;
}

nvfp4::KvPool pool_of(const nvfp4_kv_cache* c) {
    nvfp4::KvPool p;
    p.pages = c->pages;
    p.layers = c->layers;
    p.layer_stride = c->layers > 1 ? c->layer_stride : 0;
    p.page_stride = c->page_stride;
    p.record = nvfp4::kv_record_bytes(c->heads, c->head_dim, c->page_size);
    p.num_pages = (int32_t)c->num_pages;
    p.page = c->page_size;
    p.max_slots = (int32_t)c->max_slots;
    p.max_pages = c->max_pages;
    p.table = c->table;
    p.lens = c->lens;
    p.refs = c->refs;
    return p;
}

nvfp4_status check_batch(const nvfp4_kv_cache* c, int64_t layer, int64_t tokens,
                         const int32_t* cu, const int32_t* slots, int64_t seqs) {
    if (layer < 0 || layer >= c->layers) return NVFP4_ERR_ARG;
    if (tokens < 0 || tokens >= kInt32 || seqs < 0 || seqs > 65535) return NVFP4_ERR_SHAPE;
    if (tokens == 0 || seqs == 0) return NVFP4_OK;
    if (cu == nullptr) return NVFP4_ERR_NULL;
    if (!aligned(cu, 4) || !aligned(slots, 4)) return NVFP4_ERR_ALIGN;
    return NVFP4_OK;
}

// Rows [tokens, heads, dim] with element strides: 16-byte rows inside 2^56 elements.
nvfp4_status check_rows(const void* p, int esz, int64_t tokens, int64_t heads, int64_t st, int64_t sh) {
    if (st < 0 || sh < 0 || !span_ok(tokens, st) || !span_ok(heads, sh)) return NVFP4_ERR_SHAPE;
    if (p == nullptr) return NVFP4_ERR_NULL;
    if (!aligned(p, 16) || (tokens > 1 && st * esz % 16 != 0) || (heads > 1 && sh * esz % 16 != 0))
        return NVFP4_ERR_ALIGN;
    return NVFP4_OK;
}

// Positions a plan has to cover: what the caller says, and no more than the table holds.
int64_t planned_kv(const nvfp4_kv_cache* c, int64_t max_kv) {
    const int64_t cap = (int64_t)c->max_pages * c->page_size;
    return max_kv < cap ? max_kv : cap;
}

int64_t planned_q(int64_t tokens, int64_t max_q) { return max_q < tokens ? max_q : tokens; }

nvfp4_status check_attention_sizes(const nvfp4_kv_cache* c, int64_t tokens, int64_t q_heads,
                                   int64_t seqs, int64_t max_q, int64_t max_kv) {
    if (tokens < 0 || seqs < 0 || seqs > 65535 || max_q < 0 || max_kv < 0 || q_heads < 1 ||
        q_heads % c->heads != 0)
        return NVFP4_ERR_SHAPE;
    if (tokens >= kInt32 / q_heads || max_kv >= kInt32 || max_q >= kInt32 ||
        max_q * (q_heads / c->heads) >= (1 << 24))
        return NVFP4_ERR_SHAPE;
    if (!nvfp4::kv_attention_fits(c->heads, c->head_dim, tokens, q_heads, seqs, planned_q(tokens, max_q),
                                  planned_kv(c, max_kv)))
        return NVFP4_ERR_SHAPE;
    return NVFP4_OK;
}


}  // namespace

extern "C" {

size_t nvfp4_kv_page_bytes(int32_t heads, int32_t head_dim, int32_t page_size) {
    if (!layout_ok(heads, head_dim, page_size)) return 0;
    return (size_t)nvfp4::kv_record_bytes(heads, head_dim, page_size);
}

nvfp4_status nvfp4_kv_append(const nvfp4_kv_cache* cache, int64_t layer, const void* K, const void* V,
                             int dtype, int64_t tokens, int64_t stride_kt, int64_t stride_kh,
                             int64_t stride_vt, int64_t stride_vh, const int32_t* cu_tokens,
                             const int32_t* slots, int64_t seqs, int32_t lo, int32_t hi,
                             void* stream) {
    const int esz = elem_size(dtype);
    if (esz == 0) return NVFP4_ERR_DTYPE;
    if (lo > 0 || hi < 0 || lo < -125 || hi > 125) return NVFP4_ERR_WINDOW;
    nvfp4_status st = check_cache(cache, true);
    if (st != NVFP4_OK) return st;
    st = check_batch(cache, layer, tokens, cu_tokens, slots, seqs);
    if (st != NVFP4_OK) return st;
    if (tokens >= kInt32 / (cache->head_dim / 16)) return NVFP4_ERR_SHAPE;
    if (tokens == 0 || seqs == 0) return NVFP4_OK;
    st = check_rows(K, esz, tokens, cache->heads, stride_kt, stride_kh);
    if (st != NVFP4_OK) return st;
    st = check_rows(V, esz, tokens, cache->heads, stride_vt, stride_vh);
    if (st != NVFP4_OK) return st;
    if (cache->num_pages == 0 || cache->max_slots == 0 || cache->max_pages == 0) return NVFP4_OK;
    const nvfp4::KvTokens k{K, stride_kt * esz, stride_kh * esz}, v{V, stride_vt * esz, stride_vh * esz};
    const nvfp4::KvBatch b{cu_tokens, slots, (int32_t)seqs, tokens};
    return hip_status(nvfp4::launch_kv_append(view_of(cache, layer), k, v, dtype == NVFP4_DTYPE_BF16,
                                              b, lo, hi, static_cast<hipStream_t>(stream)));
}

nvfp4_status nvfp4_kv_read(const nvfp4_kv_cache* cache, int64_t layer, void* K, void* V, int dtype,
                           int64_t tokens, const int32_t* cu_tokens, const int32_t* slots,
                           int64_t seqs, void* stream) {
    if (elem_size(dtype) == 0) return NVFP4_ERR_DTYPE;
    nvfp4_status st = check_cache(cache, true);
    if (st != NVFP4_OK) return st;
    st = check_batch(cache, layer, tokens, cu_tokens, slots, seqs);
    if (st != NVFP4_OK) return st;
    if (tokens >= kInt32 / (cache->head_dim / 16)) return NVFP4_ERR_SHAPE;
    if (tokens == 0 || seqs == 0) return NVFP4_OK;
    if (K == nullptr || V == nullptr) return NVFP4_ERR_NULL;
    if (!aligned(K, 16) || !aligned(V, 16)) return NVFP4_ERR_ALIGN;
    const nvfp4::KvBatch b{cu_tokens, slots, (int32_t)seqs, tokens};
    return hip_status(nvfp4::launch_kv_read(view_of(cache, layer), K, V, dtype == NVFP4_DTYPE_BF16, b,
                                            static_cast<hipStream_t>(stream)));
}

size_t nvfp4_kv_attention_workspace_size(const nvfp4_kv_cache* cache, int dtype, int64_t tokens,
                                         int64_t q_heads, int64_t seqs, int64_t max_q,
                                         int64_t max_kv) {
    if (cache == nullptr || elem_size(dtype) == 0 ||
        !layout_ok(cache->heads, cache->head_dim, cache->page_size) || cache->max_pages < 0 ||
        check_attention_sizes(cache, tokens, q_heads, seqs, max_q, max_kv) != NVFP4_OK)
        return 0;
    return nvfp4::kv_attention_workspace_bytes(cache->heads, cache->head_dim, tokens, q_heads,
                                               seqs, planned_q(tokens, max_q),
                                               planned_kv(cache, max_kv));
}

nvfp4_status nvfp4_kv_attention(const nvfp4_kv_cache* cache, int64_t layer, const void* Q, int dtype,
                                int64_t tokens, int64_t q_heads, int64_t stride_qt,
                                int64_t stride_qh, const int32_t* cu_tokens, const int32_t* slots,
                                int64_t seqs, int64_t max_q, int64_t max_kv, float scale,
                                int causal, int64_t window, void* O, int64_t stride_ot,
                                int64_t stride_oh, float* lse, void* workspace,
                                size_t workspace_bytes, void* stream) {
    const int esz = elem_size(dtype);
    if (esz == 0) return NVFP4_ERR_DTYPE;
    nvfp4_status st = check_cache(cache, true);
    if (st != NVFP4_OK) return st;
    if (!(scale > 0.0f) || !std::isfinite(scale) || window < 0 || (window > 0 && !causal))
        return NVFP4_ERR_ARG;
    st = check_attention_sizes(cache, tokens, q_heads, seqs, max_q, max_kv);
    if (st != NVFP4_OK) return st;
    st = check_batch(cache, layer, tokens, cu_tokens, slots, seqs);
    if (st != NVFP4_OK) return st;
    if (tokens == 0 || seqs == 0 || max_q == 0) return NVFP4_OK;
    st = check_rows(Q, esz, tokens, q_heads, stride_qt, stride_qh);
    if (st != NVFP4_OK) return st;
    st = check_rows(O, esz, tokens, q_heads, stride_ot, stride_oh);
    if (st != NVFP4_OK) return st;
    const int64_t D = cache->head_dim;
    const bool by_token = (q_heads == 1 || stride_oh >= D) &&
                          (tokens == 1 || stride_ot >= (q_heads - 1) * stride_oh + D);
    const bool by_head = (tokens == 1 || stride_ot >= D) &&
                         (q_heads == 1 || stride_oh >= (tokens - 1) * stride_ot + D);
    if (!by_token && !by_head) return NVFP4_ERR_SHAPE;        // rows of O overlap
    if (!aligned(lse, 4)) return NVFP4_ERR_ALIGN;
    nvfp4::KvAttention a;
    a.kv = view_of(cache, layer);
    a.b = nvfp4::KvBatch{cu_tokens, slots, (int32_t)seqs, tokens};
    a.q = nvfp4::KvTokens{Q, stride_qt * esz, stride_qh * esz};
    a.bf16 = dtype == NVFP4_DTYPE_BF16;
    a.q_heads = (int32_t)q_heads;
    a.max_q = (int32_t)planned_q(tokens, max_q);
    a.max_kv = (int32_t)planned_kv(cache, max_kv);
    a.scale = scale;
    a.causal = causal != 0;
    a.window = window > 0x7FFFFFFF ? 0 : (int32_t)window;     // beyond every length: none
    a.out = O;
    a.out_stride_t = stride_ot * esz;
    a.out_stride_h = stride_oh * esz;
    a.lse = lse;
    a.workspace = workspace;
    const size_t need = nvfp4::kv_attention_workspace_bytes(cache->heads, D, tokens, q_heads, seqs,
                                                            a.max_q, a.max_kv);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return NVFP4_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return NVFP4_ERR_ALIGN;
    return hip_status(nvfp4::launch_kv_attention(a, static_cast<hipStream_t>(stream)));
}

size_t nvfp4_kv_pages_workspace_size(const nvfp4_kv_cache* cache, int64_t n) {
    if (cache == nullptr || cache->num_pages < 0 || cache->num_pages >= kInt32 - 4096 || n < 0 ||
        n > 65536)
        return 0;
    return nvfp4::kv_pages_workspace_bytes(cache->num_pages, n);
}

}  // extern "C"

namespace {

// Checks shared by reserve, fork and free; free has no workspace.
nvfp4_status check_pages(const nvfp4_kv_cache* cache, const int32_t* a, const int32_t* b, int64_t n,
                         const int32_t* out, bool needs_ws, const void* ws, size_t ws_bytes) {
    nvfp4_status st = check_cache(cache, false);
    if (st != NVFP4_OK) return st;
    if (n < 0 || n > 65536) return NVFP4_ERR_SHAPE;
    if (out == nullptr || (n > 0 && (a == nullptr || b == nullptr))) return NVFP4_ERR_NULL;
    if (!aligned(a, 4) || !aligned(b, 4) || !aligned(out, 4)) return NVFP4_ERR_ALIGN;
    if (needs_ws) {
        const size_t need = nvfp4::kv_pages_workspace_bytes(cache->num_pages, n);
        if (ws == nullptr || ws_bytes < need) return NVFP4_ERR_WORKSPACE;
        if (!aligned(ws, 16)) return NVFP4_ERR_ALIGN;
    }
    return NVFP4_OK;
}

}  // namespace

extern "C" {

nvfp4_status nvfp4_kv_reserve(const nvfp4_kv_cache* cache, const int32_t* slots,
                              const int32_t* counts, int64_t n, int32_t* status, void* workspace,
                              size_t workspace_bytes, void* stream) {
    const nvfp4_status st = check_pages(cache, slots, counts, n, status, true, workspace, workspace_bytes);
    if (st != NVFP4_OK) return st;
    return hip_status(nvfp4::launch_kv_reserve(pool_of(cache), slots, counts, (int32_t)n, status,
                                               workspace, static_cast<hipStream_t>(stream)));
}

nvfp4_status nvfp4_kv_fork(const nvfp4_kv_cache* cache, const int32_t* parents,
                           const int32_t* children, int64_t n, int32_t* status, void* workspace,
                           size_t workspace_bytes, void* stream) {
    const nvfp4_status st = check_pages(cache, parents, children, n, status, true, workspace, workspace_bytes);
    if (st != NVFP4_OK) return st;
    return hip_status(nvfp4::launch_kv_fork(pool_of(cache), parents, children, (int32_t)n, status,
                                            workspace, static_cast<hipStream_t>(stream)));
}

nvfp4_status nvfp4_kv_free(const nvfp4_kv_cache* cache, const int32_t* slots, int64_t n,
                           int32_t* status, void* stream) {
    const nvfp4_status st = check_pages(cache, slots, slots, n, status, false, nullptr, 0);
    if (st != NVFP4_OK) return st;
    return hip_status(nvfp4::launch_kv_free(pool_of(cache), slots, (int32_t)n, status,
                                            static_cast<hipStream_t>(stream)));
}

nvfp4_status nvfp4_kv_compact(const nvfp4_kv_cache* cache, int32_t* used, void* workspace,
                              size_t workspace_bytes, void* stream) {
    const nvfp4_status st = check_pages(cache, nullptr, nullptr, 0, used, true, workspace, workspace_bytes);
    if (st != NVFP4_OK) return st;
    return hip_status(nvfp4::launch_kv_compact(pool_of(cache), used, workspace,
                                               static_cast<hipStream_t>(stream)));
}

}  // extern "C"
