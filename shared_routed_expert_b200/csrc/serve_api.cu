// C ABI of the paged-cache, tree-attention and log-probability operators (declared
// in include/moe.h): argument validation and dispatch on the caller's stream.
#include <cmath>

#include "kernels.cuh"
#include "tree_attn.cuh"

namespace sre {

cudaError_t launch_append(const KvView& c, int head_dim, bool f8, int T, int n_q, int rot, float eps, const uint16_t* qkv,
                          long long qkv_stride, const int32_t* pos, int max_pos, const uint16_t* q_w, const uint16_t* k_w,
                          const float* cos_sin, uint16_t* q_out, long long q_stride, int32_t* bad, cudaStream_t st);
cudaError_t launch_compact(const KvView& c, int row_bytes, int n_layers, long long layer_b, const int32_t* accepted,
                           int max_accept, const int32_t* n_accepted, int32_t* bad, cudaStream_t st);
cudaError_t launch_logprobs(int T, int V, bool bf16, const void* logits, long long row_stride, const int32_t* targets,
                            int top_n, float* logprobs, float* entropy, int32_t* top_ids, float* top_lp,
                            cudaStream_t st);

namespace {

constexpr int kMaxT = 1 << 20;

bool at16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool at4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
moe_status from_cuda(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// a stride over a dimension of `size` > 1 elements: whole 16-byte steps of at least a row
bool stride_ok(int64_t stride, int64_t size, int head_dim, int esz) {
    return size <= 1 || (stride >= head_dim && stride < (int64_t{1} << 40) / esz && stride * esz % 16 == 0);
}

moe_status check_cache(const moe_kv_cache* c) {
    if (c == nullptr || !c->k || !c->v || !at16(c->k) || !at16(c->v)) return MOE_ERR_INVALID_ARG;
    if (c->num_pages <= 0 || c->n_kv <= 0 || c->page_size <= 0 || c->head_dim <= 0) return MOE_ERR_INVALID_ARG;
    if (c->dtype != MOE_BF16 && c->dtype != MOE_E4M3) return MOE_ERR_UNSUPPORTED;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return MOE_ERR_UNSUPPORTED;
    if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1))) return MOE_ERR_UNSUPPORTED;
    if (c->n_kv > 1024) return MOE_ERR_UNSUPPORTED;
    const int esz = c->dtype == MOE_BF16 ? 2 : 1;
    if (!stride_ok(c->slot_stride, c->page_size, c->head_dim, esz) || !stride_ok(c->head_stride, c->n_kv, c->head_dim, esz) ||
        !stride_ok(c->page_stride, c->num_pages, c->head_dim, esz))
        return MOE_ERR_INVALID_ARG;
    if (!(c->k_scale > 0.f) || !std::isfinite(c->k_scale) || !(c->v_scale > 0.f) || !std::isfinite(c->v_scale))
        return MOE_ERR_INVALID_ARG;
    if (c->dtype == MOE_BF16 && (c->k_scale != 1.f || c->v_scale != 1.f)) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

moe_status check_batch(const moe_kv_batch* b) {
    if (b == nullptr || b->B < 0 || b->max_new < 0 || b->max_pages < 0) return MOE_ERR_INVALID_ARG;
    if (b->B > kMaxSeqs || b->max_pages > (1 << 22) || b->max_new > kMaxT) return MOE_ERR_UNSUPPORTED;
    if (b->B == 0) return MOE_OK;
    if (b->max_pages == 0) return MOE_ERR_INVALID_ARG;
    if (!b->q_start || !b->ctx_len || !b->page_table) return MOE_ERR_INVALID_ARG;
    if (!at4(b->q_start) || !at4(b->ctx_len) || !at4(b->page_table)) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

int log2_of(int v) {
    int s = 0;
    while ((1 << s) < v) ++s;
    return s;
}

KvView view_of(const moe_kv_cache& c, const moe_kv_batch& b) {
    const long long esz = c.dtype == MOE_BF16 ? 2 : 1;
    KvView v;
    v.k = static_cast<char*>(c.k);
    v.v = static_cast<char*>(c.v);
    v.slot_b = c.slot_stride * esz;
    v.head_b = c.n_kv > 1 ? c.head_stride * esz : 0;
    v.page_b = c.num_pages > 1 ? c.page_stride * esz : 0;
    v.num_pages = c.num_pages;
    v.page_shift = log2_of(c.page_size);
    v.n_kv = c.n_kv;
    v.k_scale = c.k_scale;
    v.v_scale = c.v_scale;
    v.q_start = b.q_start;
    v.ctx_len = b.ctx_len;
    v.page_table = b.page_table;
    v.B = b.B;
    v.max_pages = b.max_pages;
    v.max_new = b.max_new;
    return v;
}

moe_status check_heads(const moe_kv_cache& c, int n_q) {
    if (n_q <= 0 || n_q % c.n_kv != 0) return MOE_ERR_INVALID_ARG;
    return n_q > 1024 ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

bool row_ok(int64_t stride, int64_t width) { return stride >= width && stride % 8 == 0 && stride < (int64_t{1} << 40); }

}  // namespace
}  // namespace sre

using namespace sre;

extern "C" {

moe_status moe_qk_norm_rope_append(const moe_kv_cache* cache, const moe_kv_batch* batch, int32_t T, int32_t n_q,
                                   int32_t rot_dim, float eps, const void* qkv, int64_t qkv_stride,
                                   const int32_t* positions, int32_t max_pos, const void* q_norm_w,
                                   const void* k_norm_w, const float* cos_sin, void* q_out, int64_t q_stride,
                                   int32_t* bad_tokens, void* stream) {
    moe_status rc = check_cache(cache);
    if (rc == MOE_OK) rc = check_batch(batch);
    if (rc == MOE_OK) rc = check_heads(*cache, n_q);
    if (rc != MOE_OK) return rc;
    if (T < 0 || !(eps >= 0.f) || !std::isfinite(eps)) return MOE_ERR_INVALID_ARG;
    if (T > kMaxT) return MOE_ERR_UNSUPPORTED;
    if (!at16(qkv) || !at16(q_out) || !at16(q_norm_w) || !at16(k_norm_w) || !at4(bad_tokens)) return MOE_ERR_INVALID_ARG;
    const int64_t d = cache->head_dim;
    if (!row_ok(qkv_stride, (n_q + 2 * cache->n_kv) * d) || !row_ok(q_stride, n_q * d)) return MOE_ERR_INVALID_ARG;
    if (!qk_norm_rope_supported(cache->head_dim, rot_dim)) return MOE_ERR_UNSUPPORTED;
    if (rot_dim > 0 && (!at4(positions) || max_pos <= 0 || !cos_sin || !at16(cos_sin))) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;                                     // (arrays of no rows may be NULL)
    if (!qkv || !q_out || (rot_dim > 0 && !positions)) return MOE_ERR_INVALID_ARG;
    if (qkv == q_out && qkv_stride != q_stride) return MOE_ERR_INVALID_ARG;
    if (batch->B == 0) return MOE_OK;
    return from_cuda(launch_append(view_of(*cache, *batch), cache->head_dim, cache->dtype == MOE_E4M3, T, n_q, rot_dim, eps,
                                   static_cast<const uint16_t*>(qkv), qkv_stride, positions, max_pos,
                                   static_cast<const uint16_t*>(q_norm_w), static_cast<const uint16_t*>(k_norm_w), cos_sin,
                                   static_cast<uint16_t*>(q_out), q_stride, bad_tokens, static_cast<cudaStream_t>(stream)));
}

size_t moe_tree_attention_workspace_size(const moe_kv_cache* cache, int32_t n_q, int32_t T) {
    if (check_cache(cache) != MOE_OK || check_heads(*cache, n_q) != MOE_OK || T < 0 || T > kMaxT) return 0;
    // partial results of the items that a cut between two blocks' shares goes through
    const size_t small = partials_bytes(kSmallBlocks, kSmallRows, cache->head_dim);
    const size_t tiles = partials_bytes(kTileBlocks, kTileRows, cache->head_dim);
    return sizeof(DevStatus) + (small > tiles ? small : tiles);
}

moe_status moe_tree_attention(const moe_kv_cache* cache, const moe_kv_batch* batch, int32_t T, int32_t n_q,
                              float softmax_scale, const void* q, int64_t q_stride, const uint64_t* tree_mask,
                              int32_t mask_words, void* out, int64_t out_stride, float* lse, void* ws,
                              size_t ws_bytes, void* stream) {
    moe_status rc = check_cache(cache);
    if (rc == MOE_OK) rc = check_batch(batch);
    if (rc == MOE_OK) rc = check_heads(*cache, n_q);
    if (rc != MOE_OK) return rc;
    const float scale_log2 = softmax_scale * cache->k_scale * kLog2E;
    if (T < 0 || !std::isfinite(scale_log2)) return MOE_ERR_INVALID_ARG;
    if (T > kMaxT) return MOE_ERR_UNSUPPORTED;
    if (!ws || !at16(q) || !at16(out) || !at4(lse) || (reinterpret_cast<uintptr_t>(ws) & 255u)) return MOE_ERR_INVALID_ARG;
    const int64_t width = static_cast<int64_t>(n_q) * cache->head_dim;
    if (!row_ok(q_stride, width) || !row_ok(out_stride, width)) return MOE_ERR_INVALID_ARG;
    if (mask_words < 0 || (tree_mask != nullptr && (mask_words < 1 || (reinterpret_cast<uintptr_t>(tree_mask) & 7u))))
        return MOE_ERR_INVALID_ARG;
    if (mask_words > 64) return MOE_ERR_UNSUPPORTED;
    if (tree_mask != nullptr && batch->max_new > 64 * mask_words) return MOE_ERR_INVALID_ARG;
    if (ws_bytes < moe_tree_attention_workspace_size(cache, n_q, T)) return MOE_ERR_WORKSPACE;
    if (T == 0) return MOE_OK;                                     // (arrays of no rows may be NULL)
    if (!q || !out || (q == out && q_stride != out_stride) || (tree_mask == nullptr && mask_words != 0)) return MOE_ERR_INVALID_ARG;
    if (batch->B == 0 || batch->max_new == 0) return MOE_OK;
    AttnArgs a;
    a.c = view_of(*cache, *batch);
    a.T = T;
    a.n_q = n_q;
    a.group = n_q / cache->n_kv;
    {   // ceil(2^(31 + s) / group) with 2^s >= group: exact for numerators below 2^31
        int s = 0;
        while ((1 << s) < a.group) ++s;
        const uint64_t mul = ((uint64_t{1} << (31 + s)) + a.group - 1) / a.group;
        a.group_mul = static_cast<uint32_t>(a.group == 1 ? 0 : mul);
        a.group_shift = s > 0 ? s - 1 : 0;
    }
    a.head_dim = cache->head_dim;
    a.f8 = cache->dtype == MOE_E4M3;
    a.scale_log2 = scale_log2;
    a.q = static_cast<const uint16_t*>(q);
    a.q_stride = q_stride;
    a.mask = tree_mask;
    a.mask_words = mask_words;
    a.out = static_cast<uint16_t*>(out);
    a.out_stride = out_stride;
    a.lse = lse;
    a.status = static_cast<DevStatus*>(ws);
    void* partials = static_cast<char*>(ws) + sizeof(DevStatus);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return from_cuda(tree_attn_wide_apply(a)    ? launch_tree_attn_wide(a, partials, st)
                     : tree_attn_tiles_apply(a) ? launch_tree_attn_tiles(a, partials, st)
                                                : launch_tree_attn_small(a, partials, st));
}

void moe_inject_attention_timeout(int n_calls) { tree_attn_inject_stall(n_calls > 0 ? n_calls : 0); }

moe_status moe_kv_compact(const moe_kv_cache* cache, const moe_kv_batch* batch, int32_t n_layers,
                          int64_t layer_stride, const int32_t* accepted, int32_t max_accept,
                          const int32_t* n_accepted, int32_t* bad_seqs, void* stream) {
    moe_status rc = check_cache(cache);
    if (rc == MOE_OK) rc = check_batch(batch);
    if (rc != MOE_OK) return rc;
    if (n_layers < 1 || max_accept < 1 || !at4(accepted) || !at4(n_accepted) || !at4(bad_seqs)) return MOE_ERR_INVALID_ARG;
    if (n_layers > 4096 || max_accept > 1024) return MOE_ERR_UNSUPPORTED;
    const int esz = cache->dtype == MOE_BF16 ? 2 : 1;
    if (!stride_ok(layer_stride, n_layers, cache->head_dim, esz)) return MOE_ERR_INVALID_ARG;
    if (batch->B == 0) return MOE_OK;                              // (arrays of no sequences may be NULL)
    if (!accepted || !n_accepted) return MOE_ERR_INVALID_ARG;
    return from_cuda(launch_compact(view_of(*cache, *batch), cache->head_dim * esz, n_layers,
                                    n_layers > 1 ? layer_stride * esz : 0, accepted, max_accept, n_accepted, bad_seqs,
                                    static_cast<cudaStream_t>(stream)));
}

moe_status moe_token_logprobs(int32_t T, int32_t V, int32_t dtype, const void* logits, int64_t row_stride,
                              const int32_t* targets, int32_t top_n, float* logprobs, float* entropy,
                              int32_t* top_ids, float* top_logprobs, void* stream) {
    if (T < 0 || V < 1 || top_n < 0 || row_stride < V) return MOE_ERR_INVALID_ARG;
    if (dtype != MOE_BF16 && dtype != MOE_F32) return MOE_ERR_UNSUPPORTED;
    if (T > kMaxT || V > (1 << 24) || top_n > 32 || row_stride >= (int64_t{1} << 40)) return MOE_ERR_UNSUPPORTED;
    if (top_n > V) return MOE_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(logits) & (dtype == MOE_BF16 ? 1u : 3u)) return MOE_ERR_INVALID_ARG;
    if (!at4(targets) || !at4(logprobs) || !at4(entropy) || !at4(top_ids) || !at4(top_logprobs)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;                                     // (arrays of no rows may be NULL)
    if (!logits) return MOE_ERR_INVALID_ARG;
    if ((targets == nullptr) != (logprobs == nullptr)) return MOE_ERR_INVALID_ARG;
    if ((top_ids == nullptr) != (top_n == 0) || (top_logprobs == nullptr) != (top_n == 0)) return MOE_ERR_INVALID_ARG;
    return from_cuda(launch_logprobs(T, V, dtype == MOE_BF16, logits, row_stride, targets, top_n, logprobs, entropy,
                                     top_ids, top_logprobs, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
