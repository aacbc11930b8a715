// Host side of the decoding-pass calls (see include/prox_decode.h): argument
// checks, workspace sizes and launches. Every step runs in the kernels of
// k_cache.cu, k_attention.cu and k_logprobs.cu.
#include "decode_internal.cuh"

#include <cmath>

#define PROX_API extern "C" __attribute__((visibility("default")))

namespace prox {
namespace {

bool aligned(const void *p, uintptr_t a = 16) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// given and aligned (lists of whole numbers and fp32 results: to 4 bytes)
bool have(const void *p, uintptr_t a = 16) { return p && aligned(p, a); }

bool shape_ok(const prox_cache *c) {
    if (!c || c->n_layers < 1 || c->n_layers > 4096 || c->n_pages < 1 || c->n_kv_heads < 1 ||
        c->n_kv_heads > 1024 || c->max_seqs < 1 || c->max_seqs > kMaxSeqs || c->max_pages < 1)
        return false;
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
        return false;
    if (c->head_dim != 64 && c->head_dim != 128) return false;
    if (c->dtype != PROX_BF16 && c->dtype != PROX_FP16) return false;
    return (long long)c->max_pages * c->page_size <= 1ll << 30 &&
           (long long)c->max_seqs * c->max_pages <= 1ll << 29 &&
           (long long)c->n_pages * c->n_kv_heads * c->page_size < 1ll << 31;
}

prox_status check_cache(const prox_cache *c) {
    if (!shape_ok(c)) return PROX_EINVAL;
    if (!have(c->k) || !have(c->v) || !have(c->page_table) || !have(c->length) || !have(c->held) ||
        !have(c->ref_count) || !have(c->free_list) || !have(c->n_free) || !have(c->status))
        return PROX_EINVAL;
    return PROX_OK;
}

bool row_stride_ok(const prox_cache *c, int heads, int64_t stride) {
    return stride % 8 == 0 && stride >= (int64_t)heads * c->head_dim && stride < 1ll << 40;
}

prox_status done(cudaError_t e) { return e == cudaSuccess ? PROX_OK : PROX_ECUDA; }

}  // namespace
}  // namespace prox

using namespace prox;

PROX_API prox_status prox_cache_init(const prox_cache *cache, void *stream) {
    prox_status ps = check_cache(cache);
    int sms;
    if (ps != PROX_OK || (ps = current_device(&sms)) != PROX_OK) return ps;
    return done(launch_cache_init(*cache, (cudaStream_t)stream));
}

PROX_API size_t prox_cache_workspace_bytes(const prox_cache *cache) {
    return shape_ok(cache) ? 16 + (size_t)cache->n_pages * 16 : 0;
}

PROX_API prox_status prox_cache_reserve(const prox_cache *cache, int n, const int32_t *seqs,
                                        const int32_t *n_new, uint8_t *ok, void *stream) {
    prox_status ps = check_cache(cache);
    if (ps != PROX_OK) return ps;
    if (n < 0 || n > cache->max_seqs) return PROX_EINVAL;
    if (n == 0) return PROX_OK;
    if (!have(seqs, 4) || !have(n_new, 4)) return PROX_EINVAL;
    int sms;
    if ((ps = current_device(&sms)) != PROX_OK) return ps;
    return done(launch_cache_reserve(*cache, n, seqs, n_new, ok, (cudaStream_t)stream));
}

PROX_API prox_status prox_cache_append(const prox_cache *cache, int layer, int n,
                                       const int32_t *seqs, const int32_t *cu_new, int rows,
                                       const uint16_t *k_new, int64_t k_stride,
                                       const uint16_t *v_new, int64_t v_stride, void *stream) {
    prox_status ps = check_cache(cache);
    if (ps != PROX_OK) return ps;
    if (layer < 0 || layer >= cache->n_layers || n < 0 || n > cache->max_seqs || rows < 0)
        return PROX_EINVAL;
    if (n == 0 || rows == 0) return PROX_OK;
    if (!have(seqs, 4) || !have(cu_new, 4) || !have(k_new) || !have(v_new)) return PROX_EINVAL;
    if (!row_stride_ok(cache, cache->n_kv_heads, k_stride) ||
        !row_stride_ok(cache, cache->n_kv_heads, v_stride))
        return PROX_EINVAL;
    int sms;
    if ((ps = current_device(&sms)) != PROX_OK) return ps;
    return done(launch_cache_append(*cache, layer, n, seqs, cu_new, rows, k_new, k_stride, v_new,
                                    v_stride, (cudaStream_t)stream));
}

PROX_API prox_status prox_cache_fork(const prox_cache *cache, int n, const int32_t *src,
                                     const int32_t *dst, int share, uint8_t *ok, void *ws,
                                     size_t ws_bytes, void *stream) {
    prox_status ps = check_cache(cache);
    if (ps != PROX_OK) return ps;
    if (n < 0 || n > cache->max_seqs || (share != 0 && share != 1)) return PROX_EINVAL;
    if (n == 0) return PROX_OK;
    if (!have(src, 4) || !have(dst, 4) || !have(ws)) return PROX_EINVAL;
    if (ws_bytes < prox_cache_workspace_bytes(cache)) return PROX_ENOMEM;
    int sms;
    if ((ps = current_device(&sms)) != PROX_OK) return ps;
    return done(launch_cache_fork(*cache, n, src, dst, share, ok, static_cast<int32_t *>(ws), sms,
                                  (cudaStream_t)stream));
}

PROX_API prox_status prox_cache_compact(const prox_cache *cache, int n, const int32_t *seqs,
                                        const int32_t *path, int max_path, const int32_t *n_path,
                                        uint8_t *ok, void *stream) {
    prox_status ps = check_cache(cache);
    if (ps != PROX_OK) return ps;
    if (n < 0 || n > cache->max_seqs || max_path < 1 || max_path > kMaxPath) return PROX_EINVAL;
    if (n == 0) return PROX_OK;
    if (!have(seqs, 4) || !have(path, 4) || !have(n_path, 4)) return PROX_EINVAL;
    int sms;
    if ((ps = current_device(&sms)) != PROX_OK) return ps;
    return done(launch_cache_compact(*cache, n, seqs, path, max_path, n_path, ok,
                                     (cudaStream_t)stream));
}

PROX_API prox_status prox_cache_free(const prox_cache *cache, int n, const int32_t *seqs,
                                     void *stream) {
    prox_status ps = check_cache(cache);
    if (ps != PROX_OK) return ps;
    if (n < 0 || n > cache->max_seqs) return PROX_EINVAL;
    if (n == 0) return PROX_OK;
    if (!have(seqs, 4)) return PROX_EINVAL;
    int sms;
    if ((ps = current_device(&sms)) != PROX_OK) return ps;
    return done(launch_cache_free(*cache, n, seqs, (cudaStream_t)stream));
}

PROX_API prox_status prox_cache_status(const prox_cache *cache, void *stream, uint32_t *flags_out) {
    prox_status ps = check_cache(cache);
    if (ps != PROX_OK) return ps;
    cudaStream_t st = (cudaStream_t)stream;
    uint32_t v = 0;
    if (cudaMemcpyAsync(&v, cache->status, sizeof v, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return PROX_ECUDA;
    // (only what was read is cleared: calls on other streams may set bits meanwhile)
    if (v && (launch_cache_clear(*cache, v, st) != cudaSuccess ||
              cudaStreamSynchronize(st) != cudaSuccess))
        return PROX_ECUDA;
    if (flags_out) *flags_out = v;
    return v & PROX_CACHE_TIMEOUT ? PROX_ETIMEOUT : v ? PROX_EDATA : PROX_OK;
}

static bool heads_ok(const prox_cache *c, int n_heads) {
    return n_heads >= 1 && n_heads % c->n_kv_heads == 0 && n_heads / c->n_kv_heads <= 64;
}

PROX_API size_t prox_attention_workspace_bytes(const prox_cache *cache, int n_heads, int max_q) {
    int sms;
    if (!shape_ok(cache) || !heads_ok(cache, n_heads) || max_q < 1 || max_q > kMaxDraft ||
        current_device(&sms) != PROX_OK)
        return 0;
    return attention_part_bytes(cache->head_dim, max_q * (n_heads / cache->n_kv_heads), sms);
}

PROX_API prox_status prox_tree_attention(const prox_cache *cache, int layer, int n,
                                         const int32_t *seqs, const int32_t *cu_q, int rows,
                                         int max_q, int n_heads, const uint16_t *q,
                                         int64_t q_stride, const uint64_t *tree, int tree_words,
                                         float scale, uint16_t *out, int64_t out_stride, float *lse,
                                         void *ws, size_t ws_bytes, void *stream) {
    prox_status ps = check_cache(cache);
    if (ps != PROX_OK) return ps;
    if (layer < 0 || layer >= cache->n_layers || n < 0 || n > 65536 || rows < 0 ||
        !heads_ok(cache, n_heads) || max_q < 1 || max_q > kMaxDraft ||
        (long long)rows * n_heads > 1ll << 31)
        return PROX_EINVAL;
    const int max_rows = max_q * (n_heads / cache->n_kv_heads);
    // (scores are kept in units of log 2, so the factor times log2(e) is used)
    const float scale_log2 = scale * 1.44269504f;
    if (!(scale > 0.f) || !std::isfinite(scale_log2)) return PROX_EINVAL;
    if (tree && (tree_words < (max_q + 63) / 64 || tree_words > 1 << 20)) return PROX_EINVAL;
    if (n == 0 || rows == 0) return PROX_OK;
    if (!have(seqs, 4) || !have(cu_q, 4) || !have(q) || !aligned(tree, 8) || !have(out) || !aligned(lse, 4) ||
        !have(ws))
        return PROX_EINVAL;
    if (!row_stride_ok(cache, n_heads, q_stride) || !row_stride_ok(cache, n_heads, out_stride))
        return PROX_EINVAL;
    int sms;
    if ((ps = current_device(&sms)) != PROX_OK) return ps;
    if (!attention_fits(*cache, max_rows)) return PROX_EINVAL;
    if (ws_bytes < attention_part_bytes(cache->head_dim, max_rows, sms)) return PROX_ENOMEM;
    const size_t one = (size_t)cache->n_pages * cache->n_kv_heads * cache->page_size * cache->head_dim;
    AttnArgs a{};
    a.cache = *cache;
    a.v_layer = cache->v + layer * one;
    a.n = n;
    a.rows = rows;
    a.max_q = max_q;
    a.n_heads = n_heads;
    a.seqs = seqs;
    a.cu_q = cu_q;
    a.q = q;
    a.q_stride = q_stride;
    a.tree = tree;
    a.tree_words = tree_words;
    a.scale_log2 = scale_log2;
    a.out = out;
    a.out_stride = out_stride;
    a.lse = lse;
    a.part = static_cast<float *>(ws);
    attention_test_state(&a.wait_us, &a.debug_skip, &a.debug_give_up);
    return done(launch_attention(a, cache->k + layer * one, max_rows, sms, (cudaStream_t)stream));
}

PROX_API prox_status prox_logprobs(int rows, int vocab, int dtype, const void *logits,
                                   int64_t stride, const int32_t *tokens, int n_tok, int top_k,
                                   float *logp, float *entropy, int32_t *top_ids, float *top_logp,
                                   void *stream) {
    if (rows < 0 || rows > 1 << 27 || vocab < 1 || vocab > 1 << 30 || n_tok < 0 || n_tok > 1024 ||
        top_k < 0 || top_k > 64 || top_k > vocab || stride < vocab || stride >= 1ll << 40)
        return PROX_EINVAL;
    if (dtype != PROX_BF16 && dtype != PROX_FP16 && dtype != PROX_FP32) return PROX_EINVAL;
    if (rows == 0) return PROX_OK;
    if (!logits || !aligned(logits, dtype == PROX_FP32 ? 4 : 2)) return PROX_EINVAL;
    if (n_tok && (!have(tokens, 4) || !have(logp, 4))) return PROX_EINVAL;
    if (top_k && (!have(top_ids, 4) || !have(top_logp, 4))) return PROX_EINVAL;
    if (!aligned(entropy, 4)) return PROX_EINVAL;
    int sms;
    prox_status ps = current_device(&sms);
    if (ps != PROX_OK) return ps;
    LogprobArgs a{rows, vocab, n_tok, top_k, logits, stride, tokens, logp, entropy, top_ids, top_logp};
    return done(launch_logprobs(a, dtype, sms, (cudaStream_t)stream));
}
