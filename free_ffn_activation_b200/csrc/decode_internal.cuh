// Internal declarations of the decoding-pass operators (include/prox_decode.h):
// kernel argument blocks and launches.
#pragma once

#include "prox_internal.cuh"
#include "prox_decode.h"

#include <cuda.h>

namespace prox {

constexpr int kMaxSeqs = 4096;      // sequences of one cache
constexpr int kMaxPath = 256;       // accepted drafted tokens of one entry
constexpr int kMaxDraft = 256;      // drafted tokens of one sequence

// page operations (k_cache.cu)
cudaError_t launch_cache_init(const prox_cache &c, cudaStream_t s);
// takes `bits` off the status word
cudaError_t launch_cache_clear(const prox_cache &c, uint32_t bits, cudaStream_t s);
cudaError_t launch_cache_reserve(const prox_cache &c, int n, const int32_t *seqs,
                                 const int32_t *n_new, uint8_t *ok, cudaStream_t s);
cudaError_t launch_cache_append(const prox_cache &c, int layer, int n, const int32_t *seqs,
                                const int32_t *cu, int rows, const uint16_t *k, int64_t k_stride,
                                const uint16_t *v, int64_t v_stride, cudaStream_t s);
cudaError_t launch_cache_fork(const prox_cache &c, int n, const int32_t *src, const int32_t *dst,
                              int share, uint8_t *ok, int32_t *ws, int sms, cudaStream_t s);
cudaError_t launch_cache_compact(const prox_cache &c, int n, const int32_t *seqs,
                                 const int32_t *path, int max_path, const int32_t *n_path,
                                 uint8_t *ok, cudaStream_t s);
cudaError_t launch_cache_free(const prox_cache &c, int n, const int32_t *seqs, cudaStream_t s);

// tree attention (k_attention.cu)
struct AttnArgs {
    alignas(64) CUtensorMap map_k, map_v;   // [rows][head_dim] of one layer
    prox_cache cache;
    const uint16_t *v_layer;                // the layer's v, for rows the tensor core must not see
    int n, rows, max_q, n_heads;
    const int32_t *seqs, *cu_q;
    const uint16_t *q;
    int64_t q_stride;
    const uint64_t *tree;
    int tree_words;
    float scale_log2;                       // the scale in units of log 2: scale * log2(e)
    uint16_t *out;
    int64_t out_stride;
    float *lse;
    float *part;                            // partial results, see k_attention.cu
    int grid;                               // CTAs of the main kernel
    uint32_t wait_us;                       // wall-clock bound of each wait, microseconds
    int debug_skip;                         // test hook: CTA 0 never loads this slot (-1: off)
    int debug_give_up;                      // test hook: its softmax does not wait for this stretch's outputs
};
// the bound of the waits and, from the test hooks, the slot not to load and the
// stretch whose outputs are not waited for (-1: none)
void attention_test_state(uint32_t *wait_us, int *skip, int *give_up);
// whether a sequence's tiles can be numbered in 31 bits
bool attention_fits(const prox_cache &c, int max_rows);
size_t attention_part_bytes(int head_dim, int max_rows, int sms);
cudaError_t launch_attention(AttnArgs &a, const uint16_t *k_layer, int max_rows, int sms,
                             cudaStream_t s);

// token log probabilities (k_logprobs.cu)
struct LogprobArgs {
    int rows, vocab, n_tok, top_k;
    const void *logits;
    int64_t stride;
    const int32_t *tokens;
    float *logp, *entropy;
    int32_t *top_ids;
    float *top_logp;
};
cudaError_t launch_logprobs(const LogprobArgs &a, int dtype, int sms, cudaStream_t s);

#ifdef __CUDACC__

// sequence of list entry i, or -1 where the entry is padding or out of range
// (then with the status bit)
__device__ __forceinline__ int entry_seq(const prox_cache &c, const int32_t *seqs, int i) {
    const int s = seqs[i];
    if (s >= 0 && s < c.max_seqs) return s;
    if (s != -1) atomicOr(c.status, PROX_CACHE_BAD_SEQ);
    return -1;
}

// committed tokens and held pages of sequence s, forced into their ranges
struct SeqState {
    int len, held;
};
__device__ __forceinline__ SeqState seq_state(const prox_cache &c, int s) {
    const int held0 = c.held[s], len0 = c.length[s];
    const int held = min(max(held0, 0), c.max_pages);
    const int len = min(max(len0, 0), held * c.page_size);
    if (held != held0 || len != len0) atomicOr(c.status, PROX_CACHE_BAD_STATE);
    return {len, held};
}

__device__ __forceinline__ bool page_ok(const prox_cache &c, int p) {
    return p >= 0 && p < c.n_pages;
}

// Bounded wait on the phase of `bar` with the given parity, for handovers of a
// microsecond: tries without a sleep hint, and looks at the clock and at `dead`
// (if there is one: a wait elsewhere in the CTA has given up) only now and then.
// False once limit_us microseconds have passed, or *dead is set.
__device__ __forceinline__ bool mbar_spin(uint64_t *bar, uint32_t parity, uint32_t limit_us,
                                          const volatile uint32_t *dead = nullptr) {
    const uint32_t addr = smem_addr(bar);
    uint64_t t0 = 0;
    for (uint32_t tries = 0;; ++tries) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(addr), "r"(parity)
            : "memory");
        if (ok) return true;
        if ((tries & 63u) == 63u) {
            const uint64_t now = global_ns();
            if (!t0) t0 = now;
            if ((dead && *dead) || now - t0 > (uint64_t)limit_us * 1000u) return false;
        }
    }
}

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

#endif  // __CUDACC__

}  // namespace prox
