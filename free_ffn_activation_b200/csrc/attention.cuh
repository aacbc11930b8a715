// What the tree-attention kernels (k_attention.cu, k_attention_tc.cu) share: the
// line of tiles that deals a ragged batch out to the CTAs, masks, packing, and
// where a cut unit's pieces lie.
#pragma once

#include "decode_internal.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

namespace prox {

constexpr int kGroup = 256;               // sequences of one launch
constexpr int kNone = (int)0x80000000;    // no page to load
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

constexpr int kKT = 64;                   // keys of a tile

// Scores in units of log 2 enter e^x as fma(score, scale, -offset) with the offset a
// rounded product itself, so the largest one comes out as the offset's rounding
// instead of 0. From this offset on that rounding (2^-24 of it: 8) would overflow
// 16-bit probabilities or lose them all, and the products are rounded first: equal
// scores then cancel exactly. Below it the exact product keeps what the scores have.
constexpr float kRoundFirst = 134217728.f;  // 2^27

#ifdef __CUDACC__

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// the line of tiles of one launch: entry i's tiles are pre[i] .. pre[i+1] - 1
// (the host keeps a launch's tiles below 2^31)
struct alignas(16) Line {
    int pre[kGroup + 1];
    int seq[kGroup], len[kGroup], tot[kGroup];   // committed, and with drafted, tokens
    int row0[kGroup], rows[kGroup];              // query rows
};

__device__ __forceinline__ int key_tiles(int tot) { return tot > 0 ? (tot + kKT - 1) / kKT : 1; }

// all threads; ROWS: rows of a row tile. Flags are raised by one CTA only.
__device__ inline void build_line(Line &ln, const AttnArgs &a, int ROWS, bool flag) {
    const prox_cache &c = a.cache;
    const int G = a.n_heads / c.n_kv_heads;
    for (int i = threadIdx.x; i < a.n; i += blockDim.x) {
        const int c0 = a.cu_q[i], c1 = a.cu_q[i + 1], s = a.seqs[i];
        const int r0 = min(max(c0, 0), a.rows);
        const int r1 = min(max(c1, r0), min(a.rows, r0 + a.max_q));
        int len = 0, tot = 0;
        uint32_t bad = r0 != c0 || r1 != c1 ? PROX_CACHE_BAD_ARG : 0u;
        if (s >= 0 && s < c.max_seqs) {
            const int held0 = c.held[s], len0 = c.length[s];
            const int held = min(max(held0, 0), c.max_pages);
            const int room = held * c.page_size;
            len = min(max(len0, 0), room);
            tot = min(len + (r1 - r0), room);
            if (held != held0 || len != len0) bad |= PROX_CACHE_BAD_STATE;
            if (tot != len + (r1 - r0)) bad |= PROX_CACHE_FULL;
        } else if (s != -1) {
            bad |= PROX_CACHE_BAD_SEQ;
        }
        if (bad && flag) atomicOr(c.status, bad);
        ln.seq[i] = s;
        ln.len[i] = len;
        ln.tot[i] = tot;
        ln.row0[i] = r0;
        ln.rows[i] = r1 - r0;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int at = 0;
        for (int b = 0; b < a.n; b += 32) {
            const int i = b + lane;
            int x = 0;
            if (i < a.n)
                x = c.n_kv_heads * ((ln.rows[i] * G + ROWS - 1) / ROWS) * key_tiles(ln.tot[i]);
            const int own = x;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (i < a.n) ln.pre[i] = at + x - own;
            at += __shfl_sync(0xffffffffu, x, 31);
        }
        if (lane == 0) ln.pre[a.n] = at;
    }
    __syncthreads();
}

// tiles of a CTA's run
__device__ __forceinline__ int run_length(const Line &ln, int n, int grid) {
    return max((int)(((unsigned)ln.pre[n] + grid - 1) / grid), 1);
}

// one stretch of a CTA's run: tiles tile0 .. tile0 + n_tiles - 1 of a unit
struct Stretch {
    int b, head, row_tile, tile0, n_tiles, all_tiles;
};
__device__ __forceinline__ Stretch stretch_at(const Line &ln, const AttnArgs &a, int ROWS, int pos,
                                              int end) {
    Stretch s;
    // last entry whose tiles begin at or before pos (pos < pre[n])
    int lo = 0, hi = a.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (ln.pre[mid] <= pos)
            lo = mid;
        else
            hi = mid - 1;
    }
    s.b = lo;
    const int G = a.n_heads / a.cache.n_kv_heads;
    const int rt = (ln.rows[s.b] * G + ROWS - 1) / ROWS;
    s.all_tiles = key_tiles(ln.tot[s.b]);
    const int local = pos - ln.pre[s.b];
    const int unit = local / s.all_tiles;
    s.tile0 = local - unit * s.all_tiles;
    s.head = unit / rt;
    s.row_tile = unit - s.head * rt;
    s.n_tiles = min(s.all_tiles - s.tile0, end - pos);
    return s;
}

// 2-D tensor-map box global -> shared, completing on an mbarrier, with an L2
// policy. Keys and values are evicted first: they are read once, and the cache
// they would fill holds the kernels' instructions, the queries, the page table
// and the pieces, whose misses each cost a microsecond of a short kernel.
__device__ __forceinline__ void box_g2s(uint32_t dst, const CUtensorMap *map, int x, int y,
                                        uint64_t *bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_addr(bar)), "l"(policy)
        : "memory");
}

// two fp32 to packed bf16 / fp16 (round to nearest even), a in the low half
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (DT == PROX_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}
template <int DT>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (DT == PROX_BF16)
        return make_float2(bf16lo(w), bf16hi(w));
    else
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
// a packed pair holds an infinity or NaN (exponent bits all set)
template <int DT>
__device__ __forceinline__ bool non_finite2(uint32_t w) {
    constexpr uint32_t E = DT == PROX_BF16 ? 0x7f80u : 0x7c00u;
    return (w & E) == E || (w & (E << 16)) == (E << 16);
}

// the pair with its infinities and NaN replaced by 0
template <int DT>
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
    constexpr uint32_t E = DT == PROX_BF16 ? 0x7f80u : 0x7c00u;
    if ((w & E) == E) w &= 0xffff0000u;
    if ((w & (E << 16)) == (E << 16)) w &= 0xffffu;
    return w;
}

// the low n bits set, any n
__device__ __forceinline__ uint64_t low_bits(int n) {
    return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull;
}

// which of the 64 keys from position w0 on row `t` of a sequence sees (bits
// of keys behind the last one are cut off by the caller)
__device__ __forceinline__ uint64_t seen_bits(const uint64_t *tree, int words, int len, int t,
                                              int w0) {
    const int c = len - w0;  // committed keys in the window
    if (!tree) return low_bits(c + t + 1);
    uint64_t bits = low_bits(c);
    if (c >= 64) return bits;
    if (c > 0) return bits | tree[0] << c;
    const int w = -c >> 6, o = -c & 63;
    if (w < words) bits |= tree[w] >> o;
    if (o && w + 1 < words) bits |= tree[w + 1] << (64 - o);
    return bits;
}

// Pieces of cut units: a CTA has at most two, slot 0 for the unit its run
// begins in and slot 1 for the one it ends in. A piece is [head_dim / 4][rows]
// float4 of unnormalised outputs (lanes that are rows write and read runs of
// 16 bytes side by side), then the rows' maxima (in log2 units) and sums.
__host__ __device__ constexpr size_t piece_floats(int dim, int rows) {
    return (size_t)rows * (dim + 2);
}
__device__ __forceinline__ float *piece(const AttnArgs &a, int cta, bool first, int dim, int rows) {
    return a.part + (size_t)(cta * 2 + (first ? 0 : 1)) * piece_floats(dim, rows);
}

#endif  // __CUDACC__

// the tensor-memory kernel with one or two row groups of 128 rows
cudaError_t launch_attention_tc(const AttnArgs &a, int row_groups, cudaStream_t s);

}  // namespace prox
