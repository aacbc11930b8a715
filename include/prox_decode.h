/*
 * prox_decode.h -- C ABI of what stands next to the sparse FFN layer in a
 * decoding pass of one to a few dozen tokens: a paged key/value cache with its
 * page operations, attention of drafted tokens over it, and the log
 * probabilities that decide which drafted tokens are kept. The Prox pages
 * describe the FFN alone and have no counterpart of these calls; their long-
 * context results (blog, "Evidence": 16K and 32K tokens) run the FFN beside
 * attention over such a cache.
 *
 * The conventions of prox.h hold (caller-owned device memory, 16-byte
 * alignment, host-checked arguments, asynchronous on `stream`), and:
 *   - Lists of whole numbers, logits and fp32 results need only the alignment
 *     of their type.
 *   - Whole numbers that live on the device (sequence lists, lengths, offsets,
 *     paths, page ids) cannot be checked on the host. The kernels check them:
 *     an entry that is out of range is left out, nothing is read or written
 *     out of bounds, and a bit of the cache's status word is set, which
 *     prox_cache_status reads.
 *   - A sequence index of -1 in a list marks a padding entry: it is left out
 *     without a status bit.
 *   - Calls that change one cache must be ordered by the caller (one stream,
 *     or events); calls that only read it (prox_tree_attention) may overlap.
 */
#ifndef PROX_DECODE_H
#define PROX_DECODE_H

#include "prox.h"

#ifdef __cplusplus
extern "C" {
#endif

/* element types */
#define PROX_BF16 0
#define PROX_FP16 1
#define PROX_FP32 2   /* logits only */

/* bits of the cache's status word */
#define PROX_CACHE_BAD_SEQ 1u    /* a sequence index out of range or listed twice      */
#define PROX_CACHE_FULL 2u       /* not enough free pages, or page table columns        */
#define PROX_CACHE_BAD_STATE 4u  /* a length, page count, page id or reference count
                                    of the cache outside its range                      */
#define PROX_CACHE_BAD_ARG 8u    /* a count, offset or path out of range, or a fork
                                    target that is not empty                            */
#define PROX_CACHE_TIMEOUT 16u   /* a bounded device-side wait gave up                  */

/*
 * A paged cache, all device pointers, caller-owned.
 *   k, v       : bf16 or fp16 [n_layers][n_pages][n_kv_heads][page_size][head_dim]:
 *                one head's rows of a page are contiguous, so a tile of keys
 *                is a few dense boxes.
 *   page_table : [max_seqs][max_pages]; row s lists the pages of sequence s,
 *                position p of it in page p / page_size; the same ids serve
 *                every layer.
 *   length     : [max_seqs] committed tokens. Drafted tokens stand behind them,
 *                at positions length, length + 1, ...
 *   held       : [max_seqs] pages the sequence holds (columns in use).
 *   ref_count  : [n_pages] sequences that hold the page; 0 = free.
 *   free_list  : [n_pages]; its first *n_free entries are the free pages. New
 *                pages are taken from its end.
 *   status     : [1] sticky PROX_CACHE_* bits.
 * Limits: page_size 16, 32, 64 or 128; head_dim 64 or 128; max_seqs <= 4096;
 * max_pages * page_size <= 2^30; max_seqs * max_pages <= 2^29;
 * n_pages * n_kv_heads * page_size < 2^31; n_kv_heads <= 1024; n_layers <= 4096.
 * A page that holds a position at or behind `length` belongs to one sequence
 * only (fork copies such a page), so appending never touches shared pages.
 */
typedef struct prox_cache {
    int n_layers, n_pages, page_size, n_kv_heads, head_dim, dtype;
    int max_seqs, max_pages;
    uint16_t *k, *v;
    int32_t *page_table, *length, *held, *ref_count, *free_list, *n_free;
    uint32_t *status;
} prox_cache;

/*
 * prox_cache_init -- empties the cache: no sequence holds a page, every page
 * is free (page 0 is taken first), status 0. k, v and the page table are left
 * as they are.
 */
prox_status prox_cache_init(const prox_cache *cache, void *stream);

/* prox_cache_workspace_bytes -- device workspace of prox_cache_fork, 0 for a
 * cache outside the limits. It needs no clearing; one call at a time uses it. */
size_t prox_cache_workspace_bytes(const prox_cache *cache);

/*
 * prox_cache_reserve -- pages for n_new more tokens behind the committed ones:
 * sequence seqs[i] holds at least ceil((length + n_new[i]) / page_size) pages
 * afterwards. Entries take pages in their order; one that finds too few free
 * pages gets none, as do those behind it that need any. One that needs more than
 * max_pages columns gets none either, and takes nothing from those behind it.
 *   seqs, n_new : device, int32 [n], 0 <= n <= max_seqs, each sequence once.
 *   ok          : device, uint8 [n], 1 = the entry has its pages, 0 = it was
 *                 refused or left out; or NULL.
 */
prox_status prox_cache_reserve(const prox_cache *cache, int n, const int32_t *seqs,
                               const int32_t *n_new, uint8_t *ok, void *stream);

/*
 * prox_cache_append -- rows of new tokens of one layer into their places:
 * rows cu_new[i] .. cu_new[i+1] - 1 of k_new and v_new go to positions
 * length, length + 1, ... of sequence seqs[i]. Pages must be there
 * (prox_cache_reserve). Lengths do not change.
 *   cu_new       : device, int32 [n + 1], ascending from 0.
 *   k_new, v_new : device, [rows][n_kv_heads][head_dim] of the cache's type,
 *                  a row k_stride (v_stride) elements behind the one before it
 *                  (a multiple of 8, at least n_kv_heads * head_dim). Rows
 *                  from cu_new[n] on have no place and are left out.
 */
prox_status prox_cache_append(const prox_cache *cache, int layer, int n, const int32_t *seqs,
                              const int32_t *cu_new, int rows, const uint16_t *k_new,
                              int64_t k_stride, const uint16_t *v_new, int64_t v_stride,
                              void *stream);

/*
 * prox_cache_fork -- sequence dst[i] becomes a copy of src[i]'s committed
 * tokens, in every layer. With share != 0 it shares src's whole pages and gets
 * a copy of the part of a page behind them; with share == 0 every page is
 * copied. Only committed rows are copied. A source may be listed several
 * times; all sources are taken as they are before the call. A target must be
 * empty (length and held 0) and listed once. Entries take pages in their
 * order, as in prox_cache_reserve; a refused target stays empty.
 *   src, dst : device, int32 [n];  ok : device, uint8 [n] or NULL.
 */
prox_status prox_cache_fork(const prox_cache *cache, int n, const int32_t *src, const int32_t *dst,
                            int share, uint8_t *ok, void *ws, size_t ws_bytes, void *stream);

/*
 * prox_cache_compact -- keeps the accepted path of a drafted tree: for entry i
 * the drafted rows path[i][0] < path[i][1] < ... (n_path[i] of them, counted
 * from the first drafted row) move to positions length, length + 1, ... in
 * every layer, and length grows by n_path[i]. Pages stay with the sequence.
 *   path   : device, int32 [n][max_path], 1 <= max_path <= 256.
 *   n_path : device, int32 [n], 0 <= n_path[i] <= max_path.
 *   ok     : device, uint8 [n] or NULL; an entry whose path is not strictly
 *            ascending, leaves the held pages or meets a page id out of range is
 *            refused as a whole.
 */
prox_status prox_cache_compact(const prox_cache *cache, int n, const int32_t *seqs,
                               const int32_t *path, int max_path, const int32_t *n_path,
                               uint8_t *ok, void *stream);

/*
 * prox_cache_free -- gives back all pages of the listed sequences; their
 * length and held become 0. A page that no sequence holds any more goes to
 * the end of the free list, in the order in which the entries list the pages.
 */
prox_status prox_cache_free(const prox_cache *cache, int n, const int32_t *seqs, void *stream);

/*
 * prox_cache_status -- reads the cache's status word and clears the bits that it
 * returns (synchronises `stream`; a bit that a call on another stream sets
 * meanwhile is returned now or by the next call). PROX_ETIMEOUT if a wait gave up since the last read, else
 * PROX_EDATA if another bit was set, else PROX_OK; *flags_out (host, may be NULL) receives the bits.
 */
prox_status prox_cache_status(const prox_cache *cache, void *stream, uint32_t *flags_out);

/*
 * prox_tree_attention -- attention of drafted tokens over one layer of the
 * cache, with grouped heads. Query row r = cu_q[i] + t is drafted token t of
 * sequence s = seqs[i]; with L = length[s] and T = cu_q[i+1] - cu_q[i] it sees
 * the keys j < L and those drafted keys L + d, d < T, whose bit is set:
 *   tree == NULL : d <= t (a chain: an ordinary decoding step for T = 1);
 *   else         : bit d % 64 of tree[r][d / 64] (its ancestors and itself).
 *   out[r][h] = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j - m),
 *   lse[r][h] = log sum_j exp(scale q.k_j)   (natural log),
 * with q and keys of head h and key/value head h / (n_heads / n_kv_heads).
 * A row that sees no key (and every row of an entry that is left out) gets
 * out 0 and lse -inf; what a masked key or value
 * holds (NaN and infinities among it) has no influence. An infinite value that
 * is seen counts p_j v_j as any other: an infinity, or NaN where p_j is 0. That
 * is where it underflows in fp32 for a drafted token, and in the cache's type
 * for a committed one; close to it, which of the two comes out may depend on how
 * the keys were divided among the blocks.
 * The drafted rows must be in the cache already (prox_cache_append). Rows
 * behind cu_q[n] are neither read nor written.
 *   q    : device, [rows][n_heads][head_dim] of the cache's type, rows
 *          q_stride elements apart (a multiple of 8, >= n_heads * head_dim).
 *   cu_q : device, int32 [n + 1], ascending from 0; no sequence has more than
 *          max_q rows (1 <= max_q <= 256).
 *   tree : device, uint64 [rows][tree_words] or NULL; tree_words >=
 *          ceil(max_q / 64). Bits d >= T are ignored.
 *   scale: > 0; scale * log2(e), and the scores times that, finite in fp32.
 *   out  : device, the cache's type, [rows][n_heads][head_dim], rows
 *          out_stride elements apart (as q_stride).
 *   lse  : device, fp32 [rows][n_heads], or NULL.
 *   ws   : device, prox_attention_workspace_bytes(...) bytes, needs no
 *          clearing; calls that overlap on the device need one each.
 * Arithmetic: scores, softmax statistics and sums in fp32; the probabilities
 * are rounded to the cache's type for the product with v. The sums are divided
 * at the end: |v| * 2^8 * (keys that a row sees) has to stay below 2^128.
 * `out` may be `q` itself (the same rows); otherwise no output overlaps what
 * the call reads.
 * A sequence may be listed several times. n <= 65536, n_heads a multiple of
 * n_kv_heads, n_heads <= 64 * n_kv_heads; n_kv_heads * (max_pages * page_size
 * / 64 + 1) < 2^31 / 64.
 */
size_t prox_attention_workspace_bytes(const prox_cache *cache, int n_heads, int max_q);
prox_status prox_tree_attention(const prox_cache *cache, int layer, int n, const int32_t *seqs,
                                const int32_t *cu_q, int rows, int max_q, int n_heads,
                                const uint16_t *q, int64_t q_stride, const uint64_t *tree,
                                int tree_words, float scale, uint16_t *out, int64_t out_stride,
                                float *lse, void *ws, size_t ws_bytes, void *stream);

/*
 * prox_logprobs -- log probabilities under softmax of a row of logits:
 *   logp[r][i]     = x[tokens[r][i]] - log sum_v exp(x[v]);
 *   entropy[r]     = -sum_v p_v log p_v (natural log);
 *   top_ids[r][i], top_logp[r][i] : the top_k largest logits in descending
 *                    order, of equal ones the lower index first.
 * A logit of -inf has probability 0; a row of nothing else has logp -inf and
 * entropy 0. NaN or +inf in a row makes its logp, top_logp and entropy NaN
 * (top_ids then list NaN first). A token outside [0, vocab) gets logp NaN.
 *   logits : device, dtype PROX_BF16, PROX_FP16 or PROX_FP32, [rows][vocab],
 *            rows `stride` elements apart (>= vocab), aligned to its type only.
 *   tokens : device, int32 [rows][n_tok], 0 <= n_tok <= 1024 (NULL if 0).
 *   logp   : device, fp32 [rows][n_tok];  entropy : device, fp32 [rows] or NULL.
 *   top_ids, top_logp : device, int32 / fp32 [rows][top_k],
 *            0 <= top_k <= min(64, vocab) (NULL if 0).
 * Sums in fp32 per thread (of up to vocab / 256 terms, so off by 2^-24 for each
 * at most) and in fp64 across threads, in a fixed order.
 */
prox_status prox_logprobs(int rows, int vocab, int dtype, const void *logits, int64_t stride,
                          const int32_t *tokens, int n_tok, int top_k, float *logp, float *entropy,
                          int32_t *top_ids, float *top_logp, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PROX_DECODE_H */
