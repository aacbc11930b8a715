// Attention of drafted tokens over the paged cache (include/prox_decode.h).
//
// With the grouped heads of one key/value head and the drafted tokens of one
// sequence as rows, x = scale q k^T over all keys, a row's result is
//   o = sum_j e^(x_j - m) v_j / sum_j e^(x_j - m),   m = max_j x_j,
// taken in one pass over the keys with a running maximum and sum. Few rows
// read a long cache, so the bytes of k and v bound it, and each is read once.
//
// Work is a line of tiles: for every sequence, key/value head and tile of
// rows (a unit) the tiles of 64 keys one after another. Each CTA computes the
// line from the sequences' lengths and takes an equal run of it, so ragged
// batches are balanced without the host knowing the lengths. A unit that lies
// in one CTA's run is written at once; one that is cut leaves its pieces'
// maxima, sums and unnormalised outputs in the workspace, and a second kernel
// joins them in a fixed order.
//
// In a CTA one warp loads: tensor-map boxes of one page's rows and 64 elements,
// 128-byte swizzled, into a ring of stages on mbarriers. Four warps compute
// with mma.sync m16n8k16 (bf16 or fp16, fp32 sums): up to 64 rows the tensor
// pipes keep up with the memory, and a warp's registers carry a tile of
// scores straight into the second product.
#include "decode_internal.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace prox {
namespace {

constexpr int kKT = 64;             // keys of a tile
constexpr int kGroup = 256;         // sequences of one launch
constexpr int kWarps = 4;           // computing warps
constexpr int kThreads = 32 * kWarps + 32;
constexpr int kMaxStages = 8;
constexpr int kNone = (int)0x80000000;   // no page to load
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// the line of tiles of one launch: entry i's tiles are pre[i] .. pre[i+1] - 1
struct Line {
    long long pre[kGroup + 1];
    int seq[kGroup], len[kGroup], tot[kGroup];   // committed, and with drafted, tokens
    int row0[kGroup], rows[kGroup];              // query rows
};

__device__ __forceinline__ int key_tiles(int tot) { return tot > 0 ? (tot + kKT - 1) / kKT : 1; }

// all threads; ROWS: rows of a row tile. Flags are raised by one CTA only.
__device__ void build_line(Line &ln, const AttnArgs &a, int ROWS, bool flag) {
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
        long long at = 0;
        for (int b = 0; b < a.n; b += 32) {
            const int i = b + lane;
            long long x = 0;
            if (i < a.n)
                x = (long long)c.n_kv_heads * ((ln.rows[i] * G + ROWS - 1) / ROWS) *
                    key_tiles(ln.tot[i]);
            const long long own = x;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, x, o);
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
__device__ __forceinline__ long long run_length(const Line &ln, int n, int grid) {
    return max((ln.pre[n] + grid - 1) / grid, 1LL);
}

// last entry whose tiles begin at or before pos (pos < pre[n])
__device__ __forceinline__ int entry_at(const Line &ln, int n, long long pos) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (ln.pre[mid] <= pos)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// one stretch of a CTA's run: tiles tile0 .. tile0 + n_tiles - 1 of a unit
struct Stretch {
    int b, head, row_tile, tile0, n_tiles, all_tiles;
};
__device__ __forceinline__ Stretch stretch_at(const Line &ln, const AttnArgs &a, int ROWS,
                                              long long pos, long long end) {
    Stretch s;
    s.b = entry_at(ln, a.n, pos);
    const int G = a.n_heads / a.cache.n_kv_heads;
    const int rt = (ln.rows[s.b] * G + ROWS - 1) / ROWS;
    s.all_tiles = key_tiles(ln.tot[s.b]);
    const long long local = pos - ln.pre[s.b];
    const int unit = (int)(local / s.all_tiles);
    s.tile0 = (int)(local - (long long)unit * s.all_tiles);
    s.head = unit / rt;
    s.row_tile = unit - s.head * rt;
    s.n_tiles = (int)min((long long)(s.all_tiles - s.tile0), end - pos);
    return s;
}

// 2-D tensor-map box global -> shared, completing on an mbarrier
__device__ __forceinline__ void box_g2s(uint32_t dst, const CUtensorMap *map, int x, int y,
                                        uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

template <int DT>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    if constexpr (DT == PROX_BF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

template <int D, int RG>
struct Cfg {
    static constexpr int KG = kWarps / RG;        // key groups
    static constexpr int WK = kKT / KG;           // keys of a tile one warp takes
    static constexpr int ROWS = 16 * RG;
    static constexpr int NST = D == 128 ? 3 : 6;  // ring stages
    static constexpr int HALF = kKT * 128;        // bytes of 64 elements of a tile's rows
    static constexpr int TILE = HALF * (D / 64);  // bytes of a tile of k (or v)
    static constexpr int OBUF = 16 * D * 4 / 2;   // half of a warp's outputs
};

struct Ctl {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t poison;              // drafted keys of the tile whose v is not finite
    uint32_t bad[kMaxStages];     // pages of the stage's tile with an id out of range
    float m[kWarps * 16], l[kWarps * 16];
};

template <int D, int RG>
constexpr size_t smem_bytes() {
    using C = Cfg<D, RG>;
    return 1024 + (size_t)C::NST * 2 * C::TILE + 2 * C::OBUF + sizeof(Line) + sizeof(Ctl);
}

__device__ __forceinline__ bool bar_or(bool p) {  // over the computing warps
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %1, 0;\n\t"
        "bar.red.or.pred q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)p)
        : "memory");
    return r != 0;
}

template <int D, int DT, int RG>
__global__ void __launch_bounds__(kThreads, 2) k_attention(const __grid_constant__ AttnArgs a) {
    using C = Cfg<D, RG>;
    constexpr int KG = C::KG, WK = C::WK, ROWS = C::ROWS, NST = C::NST;
    constexpr int NB = WK / 8, DB = D / 8;
    extern __shared__ unsigned char raw[];
    unsigned char *sm = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    float4 *obuf = reinterpret_cast<float4 *>(sm + NST * 2 * C::TILE);
    Line &ln = *reinterpret_cast<Line *>(sm + NST * 2 * C::TILE + 2 * C::OBUF);
    Ctl &ctl = *reinterpret_cast<Ctl *>(&ln + 1);
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const prox_cache &c = a.cache;
    const int ps = c.page_size, G = a.n_heads / c.n_kv_heads;

    if (tid == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(&ctl.full[i], 1);
            mbar_init(&ctl.empty[i], kWarps);
        }
        ctl.poison = 0;
        mbar_fence_init();
    }
    pdl_wait();
    pdl_launch();
    build_line(ln, a, ROWS, blockIdx.x == 0);  // (its barriers cover the mbarriers too)
    const long long run = run_length(ln, a.n, a.grid);
    const long long begin = blockIdx.x * run, end = min(begin + run, ln.pre[a.n]);
    if (begin >= end) return;
    const int per_box = min(ps, kKT);           // rows of a box
    const int boxes = kKT / per_box;            // pages of a tile

    if (wid == kWarps) {
        // ------------------------------------------------------------------
        // loading warp: lane = (page of the tile, k or v, 64 elements)
        // ------------------------------------------------------------------
        constexpr int H = D / 64;
        const int pg = lane / (2 * H), kv = lane / H & 1, half = lane % H;
        bool live = true;
        int it = 0;
        for (long long pos = begin; pos < end;) {
            const Stretch st = stretch_at(ln, a, ROWS, pos, end);
            pos += st.n_tiles;
            const int tot = ln.tot[st.b];
            const int32_t *table = c.page_table + (size_t)max(ln.seq[st.b], 0) * c.max_pages;
            auto page_of = [&](int tile) {
                const int key = tile * kKT + pg * per_box;
                return pg < boxes && key < tot ? table[key / ps] : kNone;
            };
            int page = page_of(st.tile0);
            for (int i = 0; i < st.n_tiles; ++i, ++it) {
                const int tile = st.tile0 + i, slot = it % NST;
                const int next = i + 1 < st.n_tiles ? page_of(tile + 1) : kNone;
                if (it >= NST && live && !mbar_wait(&ctl.empty[slot], (it / NST - 1) & 1, a.wait_us)) {
                    live = false;
                    if (lane == 0) atomicOr(c.status, PROX_CACHE_TIMEOUT);
                }
                if (!live) break;
                // a page id out of range: zeros (a box outside the map), and the mask
                const bool wanted = page != kNone, good = page >= 0 && page < c.n_pages;
                const unsigned bad = __ballot_sync(0xffffffffu, wanted && !good);
                const unsigned load = __ballot_sync(0xffffffffu, wanted);
                if (lane == 0) {
                    uint32_t pages = 0;
                    for (int p = 0; p < boxes; ++p) pages |= (bad >> (p * 2 * H) & 1u) << p;
                    if (pages) atomicOr(c.status, PROX_CACHE_BAD_STATE);
                    ctl.bad[slot] = pages;
                    mbar_arrive_expect_tx(&ctl.full[slot], __popc(load) * per_box * 128);
                }
                __syncwarp();
                if (wanted) {
                    const int y = good ? (page * c.n_kv_heads + st.head) * ps + tile * kKT % ps
                                       : c.n_pages * c.n_kv_heads * ps;
                    box_g2s(smem_addr(sm) + slot * 2 * C::TILE + kv * C::TILE + half * C::HALF +
                                pg * per_box * 128,
                            kv ? &a.map_v : &a.map_k, half * 64, y, &ctl.full[slot]);
                }
                page = next;
            }
            if (!live) break;
        }
        // after a wait that gave up: let the copies in flight land
        if (!live)
            for (int k = max(0, it - NST); k < it; ++k)
                mbar_wait(&ctl.full[k % NST], (k / NST) & 1, 1000);
        return;
    }

    // ----------------------------------------------------------------------
    // computing warps
    // ----------------------------------------------------------------------
    const int rg = wid % RG, kg = wid / RG, g = lane >> 2, tg = lane & 3;
    const float sc = a.scale * kLog2e;
    bool live = true;
    int it = 0;
    for (long long pos = begin; pos < end;) {
        const Stretch st = stretch_at(ln, a, ROWS, pos, end);
        const bool first = pos == begin;
        pos += st.n_tiles;
        const int len = ln.len[st.b], tot = ln.tot[st.b];
        const int n_rows = ln.rows[st.b] * G;     // rows of this key/value head
        // this thread's two rows: drafted token, head, and whether they exist
        int tok[2];
        const uint16_t *qp[2];
        bool there[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = st.row_tile * ROWS + rg * 16 + g + 8 * e;
            there[e] = r < n_rows;
            tok[e] = there[e] ? r / G : 0;
            qp[e] = a.q + (size_t)(ln.row0[st.b] + tok[e]) * a.q_stride +
                    (size_t)(st.head * G + (there[e] ? r - tok[e] * G : 0)) * D;
        }
        uint32_t qf[D / 16][4];
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint16_t *p = qp[e] + k * 16 + tg * 2;
                qf[k][e] = there[e] ? *reinterpret_cast<const uint32_t *>(p) : 0u;
                qf[k][2 + e] = there[e] ? *reinterpret_cast<const uint32_t *>(p + 8) : 0u;
            }
        float o[DB][4];
#pragma unroll
        for (int d = 0; d < DB; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

        for (int i = 0; i < st.n_tiles; ++i, ++it) {
            const int tile = st.tile0 + i, slot = it % NST;
            if (live && !mbar_wait(&ctl.full[slot], (it / NST) & 1, a.wait_us)) {
                live = false;
                if (lane == 0) atomicOr(c.status, PROX_CACHE_TIMEOUT);
            }
            const uint32_t sk = smem_addr(sm) + slot * 2 * C::TILE, sv = sk + C::TILE;
            const uint32_t bad = ctl.bad[slot];
            // tiles with drafted or missing keys have rows of v that must not
            // meet the tensor core (0 * inf is not 0); these tiles and those
            // with unreadable pages have a mask
            const bool edge = (tile + 1) * kKT > len, masked = edge || bad;
            uint64_t seen[2] = {~0ull, ~0ull}, poison = 0;
            const uint64_t valid = low_bits(tot - tile * kKT);
            if (edge) {
                // two threads a row: zero it if it is not valid, else look for
                // infinities and NaN (drafted rows only: every row sees the others)
                const int row = tid >> 1;
                unsigned char *vr = sm + slot * 2 * C::TILE + C::TILE + row * 128;
                bool odd = false;
                if (!(valid >> row & 1)) {
                    for (int x = tid & 1; x < D / 8; x += 2)
                        *reinterpret_cast<uint4 *>(vr + (x >> 3) * C::HALF + (x & 7) * 16) =
                            make_uint4(0, 0, 0, 0);
                } else if (tile * kKT + row >= len) {
                    for (int x = tid & 1; x < D / 8; x += 2) {
                        const uint4 w =
                            *reinterpret_cast<const uint4 *>(vr + (x >> 3) * C::HALF + (x & 7) * 16);
                        odd |= non_finite2<DT>(w.x) || non_finite2<DT>(w.y) ||
                               non_finite2<DT>(w.z) || non_finite2<DT>(w.w);
                    }
                }
                if (bar_or(odd)) {
                    if (odd)
                        atomicOr(reinterpret_cast<unsigned long long *>(&ctl.poison), 1ull << row);
                    named_bar_sync(1, 128);
                    poison = ctl.poison;
                    if (poison >> row & 1)
                        for (int x = tid & 1; x < D / 8; x += 2)
                            *reinterpret_cast<uint4 *>(vr + (x >> 3) * C::HALF + (x & 7) * 16) =
                                make_uint4(0, 0, 0, 0);
                    named_bar_sync(1, 128);
                    if (tid == 0) ctl.poison = 0;
                }
                // the stage is refilled by the async proxy
                fence_proxy_async_smem();
            }
            if (masked) {
                uint64_t readable = valid;
                for (int p = 0; p < boxes; ++p)
                    if (bad >> p & 1) readable &= ~(low_bits(per_box) << (p * per_box));
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int w0 = tile * kKT + kg * WK;
                    const uint64_t *tr =
                        a.tree ? a.tree + (size_t)(ln.row0[st.b] + tok[e]) * a.tree_words : nullptr;
                    seen[e] = there[e] ? seen_bits(tr, a.tree_words, len, tok[e], w0) &
                                             (readable >> (kg * WK))
                                       : 0ull;
                }
            }

            // scores of 16 rows and WK keys
            float s[NB][4];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) s[nb][0] = s[nb][1] = s[nb][2] = s[nb][3] = 0.f;
#pragma unroll
            for (int nb = 0; nb < NB; nb += 2) {
                // lanes 0-7, 8-15: keys 0-7 at elements 0, 8; 16-31: keys 8-15
                const int key = kg * WK + nb * 8 + (lane & 7) + (lane >> 4) * 8;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const int ch = k * 2 + (lane >> 3 & 1);
                    uint32_t b[4];
                    ldsm4(b, sk + (ch >> 3) * C::HALF + key * 128 + (((ch & 7) ^ (key & 7)) << 4));
                    mma16816<DT>(s[nb], qf[k], b[0], b[1]);
                    mma16816<DT>(s[nb + 1], qf[k], b[2], b[3]);
                }
            }
            if (masked) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        if (!(seen[x >> 1] >> (nb * 8 + tg * 2 + (x & 1)) & 1)) s[nb][x] = -INFINITY;
            }
            float mu[2], r[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float mx = -INFINITY;
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) mx = fmaxf(mx, fmaxf(s[nb][2 * e], s[nb][2 * e + 1]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float nm = fmaxf(m[e], mx * sc);
                // a row that has seen nothing yet: any finite offset will do
                mu[e] = nm == -INFINITY ? 0.f : nm;
                r[e] = nm > m[e] ? ex2(m[e] - mu[e]) : 1.f;
                l[e] *= r[e];
                m[e] = nm;
            }
            if (__any_sync(0xffffffffu, r[0] != 1.f || r[1] != 1.f)) {
#pragma unroll
                for (int d = 0; d < DB; ++d) {
                    o[d][0] *= r[0];
                    o[d][1] *= r[0];
                    o[d][2] *= r[1];
                    o[d][3] *= r[1];
                }
            }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    s[nb][x] = ex2(fmaf(s[nb][x], sc, -mu[x >> 1]));
                    l[x >> 1] += s[nb][x];
                }
            // outputs += probabilities x v
#pragma unroll
            for (int k = 0; k < WK / 16; ++k) {
                const uint32_t p[4] = {
                    pack2<DT>(s[2 * k][0], s[2 * k][1]), pack2<DT>(s[2 * k][2], s[2 * k][3]),
                    pack2<DT>(s[2 * k + 1][0], s[2 * k + 1][1]),
                    pack2<DT>(s[2 * k + 1][2], s[2 * k + 1][3])};
                // lanes 0-7, 8-15: keys 0-7, 8-15 at element 0; 16-31: at element 8
                const int key = kg * WK + k * 16 + (lane & 15);
#pragma unroll
                for (int d = 0; d < DB; d += 2) {
                    const int ch = d + (lane >> 4);
                    uint32_t b[4];
                    ldsm4t(b, sv + (ch >> 3) * C::HALF + key * 128 + (((ch & 7) ^ (key & 7)) << 4));
                    mma16816<DT>(o[d], p, b[0], b[1]);
                    mma16816<DT>(o[d + 1], p, b[2], b[3]);
                }
            }
            if (poison) {
                // drafted rows of v with infinities or NaN, for the rows that see them
                for (uint64_t w = poison >> (kg * WK) & low_bits(WK); w; w &= w - 1) {
                    const int j = __ffsll((long long)w) - 1;
                    float p0 = 0.f, p1 = 0.f;
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
                        if (nb == j >> 3) {
                            p0 = j & 1 ? s[nb][1] : s[nb][0];
                            p1 = j & 1 ? s[nb][3] : s[nb][2];
                        }
                    p0 = __shfl_sync(0xffffffffu, p0, (lane & 28) | (j >> 1 & 3));
                    p1 = __shfl_sync(0xffffffffu, p1, (lane & 28) | (j >> 1 & 3));
                    const int key = tile * kKT + kg * WK + j;
                    const int page = c.page_table[(size_t)ln.seq[st.b] * c.max_pages + key / ps];
                    if (!page_ok(c, page)) continue;  // (cannot be: its box was read)
                    const uint16_t *v =
                        a.v_layer + (((size_t)page * c.n_kv_heads + st.head) * ps + key % ps) * D;
#pragma unroll
                    for (int d = 0; d < DB; ++d) {
                        const float2 x =
                            unpack2<DT>(*reinterpret_cast<const uint32_t *>(v + d * 8 + tg * 2));
                        if (seen[0] >> j & 1) {
                            o[d][0] += p0 * x.x;
                            o[d][1] += p0 * x.y;
                        }
                        if (seen[1] >> j & 1) {
                            o[d][2] += p1 * x.x;
                            o[d][3] += p1 * x.y;
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.empty[slot]);
        }

        // ------------------------------------------------------------------
        // join the key groups, then write the rows or leave a piece
        // ------------------------------------------------------------------
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
        }
        if constexpr (KG > 1) {
            if (tg == 0) {
                ctl.m[wid * 16 + g] = m[0];
                ctl.m[wid * 16 + g + 8] = m[1];
                ctl.l[wid * 16 + g] = l[0];
                ctl.l[wid * 16 + g + 8] = l[1];
            }
            named_bar_sync(1, 128);
            float f[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float M = -INFINITY, sum = 0.f;
                for (int k = 0; k < KG; ++k) M = fmaxf(M, ctl.m[(k * RG + rg) * 16 + g + 8 * e]);
                const float mu = M == -INFINITY ? 0.f : M;
                for (int k = 0; k < KG; ++k) {
                    const int w = (k * RG + rg) * 16 + g + 8 * e;
                    sum += ex2(ctl.m[w] - mu) * ctl.l[w];
                }
                f[e] = ex2(m[e] - mu);
                m[e] = M;
                l[e] = sum;
            }
#pragma unroll
            for (int d = 0; d < DB; ++d) {
                o[d][0] *= f[0];
                o[d][1] *= f[0];
                o[d][2] *= f[1];
                o[d][3] *= f[1];
            }
            // pairs of key groups, half of the columns at a time
#pragma unroll
            for (int hop = 1; hop < KG; hop *= 2)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float4 *buf = obuf + ((kg / (2 * hop)) * RG + rg) % 2 * (C::OBUF / 16);
                    named_bar_sync(1, 128);
                    if (kg % (2 * hop) == hop)
#pragma unroll
                        for (int d = 0; d < DB / 2; ++d)
                            buf[d * 32 + lane] = make_float4(
                                o[h * DB / 2 + d][0], o[h * DB / 2 + d][1], o[h * DB / 2 + d][2],
                                o[h * DB / 2 + d][3]);
                    named_bar_sync(1, 128);
                    if (kg % (2 * hop) == 0)
#pragma unroll
                        for (int d = 0; d < DB / 2; ++d) {
                            const float4 v = buf[d * 32 + lane];
                            o[h * DB / 2 + d][0] += v.x;
                            o[h * DB / 2 + d][1] += v.y;
                            o[h * DB / 2 + d][2] += v.z;
                            o[h * DB / 2 + d][3] += v.w;
                        }
                }
        }
        if (kg == 0) {
            if (st.n_tiles == st.all_tiles) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (!there[e]) continue;
                    const int r = st.row_tile * ROWS + rg * 16 + g + 8 * e;
                    const int head = st.head * G + r - tok[e] * G;
                    const size_t row = ln.row0[st.b] + tok[e];
                    const float inv = l[e] == 0.f ? 0.f : 1.f / l[e];
                    uint16_t *op = a.out + row * a.out_stride + (size_t)head * D + tg * 2;
#pragma unroll
                    for (int d = 0; d < DB; ++d)
                        *reinterpret_cast<uint32_t *>(op + d * 8) =
                            pack2<DT>(o[d][2 * e] * inv, o[d][2 * e + 1] * inv);
                    if (a.lse && tg == 0)
                        a.lse[row * a.n_heads + head] =
                            m[e] == -INFINITY && l[e] == 0.f ? -INFINITY
                                                             : (m[e] + log2f(l[e])) * kLn2;
                }
            } else {
                float *part = a.part + (size_t)(blockIdx.x * 2 + (first ? 0 : 1)) * ROWS * (D + 2);
                float *pm = part + ROWS * D;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = rg * 16 + g + 8 * e;
#pragma unroll
                    for (int d = 0; d < DB; ++d)
                        *reinterpret_cast<float2 *>(part + (size_t)r * D + d * 8 + tg * 2) =
                            make_float2(o[d][2 * e], o[d][2 * e + 1]);
                    if (tg == 0) {
                        pm[r] = m[e];
                        pm[ROWS + r] = l[e];
                    }
                }
            }
        }
        if constexpr (KG > 1) named_bar_sync(1, 128);  // ctl.m and obuf are free again
    }
}

// Joins the pieces of units that were cut: one warp an output row, the pieces
// in the order of the line.
template <int D, int DT>
__global__ void __launch_bounds__(256) k_attention_join(const __grid_constant__ AttnArgs a, int ROWS) {
    __shared__ Line ln;
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    pdl_wait();
    pdl_launch();
    build_line(ln, a, ROWS, false);
    const long long id = (long long)blockIdx.x * 8 + wid;
    const int row = (int)(id / a.n_heads), head = (int)(id - (long long)row * a.n_heads);
    if (row >= a.rows) return;
    int b = -1;
    for (int i0 = 0; i0 < a.n; i0 += 32) {
        const int i = i0 + lane;
        const bool in = i < a.n && row >= ln.row0[i] && row < ln.row0[i] + ln.rows[i];
        const unsigned who = __ballot_sync(0xffffffffu, in);
        if (who && b < 0) b = i0 + __ffs(who) - 1;
    }
    if (b < 0) return;
    const int G = a.n_heads / a.cache.n_kv_heads;
    const int r = (row - ln.row0[b]) * G + head % G;
    const int rt = (ln.rows[b] * G + ROWS - 1) / ROWS, kt = key_tiles(ln.tot[b]);
    const long long run = run_length(ln, a.n, a.grid);
    const long long u0 = ln.pre[b] + ((long long)(head / G) * rt + r / ROWS) * kt, u1 = u0 + kt;
    const long long c0 = u0 / run, c1 = (u1 - 1) / run;
    if (c0 == c1) return;  // written by its CTA
    const int rr = r % ROWS;
    constexpr int V = D / 32;
    float o[V] = {}, m = -INFINITY, l = 0.f;
    for (long long cta = c0; cta <= c1; ++cta) {
        const float *part = a.part + (size_t)(cta * 2 + (cta * run >= u0 ? 0 : 1)) * ROWS * (D + 2);
        const float pm = part[ROWS * D + rr], pl = part[ROWS * D + ROWS + rr];
        float x[V];
        if constexpr (V == 4) {
            const float4 v = *reinterpret_cast<const float4 *>(part + (size_t)rr * D + lane * 4);
            x[0] = v.x;
            x[1] = v.y;
            x[2] = v.z;
            x[3] = v.w;
        } else {
            const float2 v = *reinterpret_cast<const float2 *>(part + (size_t)rr * D + lane * 2);
            x[0] = v.x;
            x[1] = v.y;
        }
        const float nm = fmaxf(m, pm), mu = nm == -INFINITY ? 0.f : nm;
        const float f0 = ex2(m - mu), f1 = ex2(pm - mu);
        l = l * f0 + pl * f1;
#pragma unroll
        for (int k = 0; k < V; ++k) o[k] = o[k] * f0 + x[k] * f1;
        m = nm;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint16_t *op = a.out + (size_t)row * a.out_stride + (size_t)head * D + lane * V;
    if constexpr (V == 4)
        *reinterpret_cast<uint2 *>(op) =
            make_uint2(pack2<DT>(o[0] * inv, o[1] * inv), pack2<DT>(o[2] * inv, o[3] * inv));
    else
        *reinterpret_cast<uint32_t *>(op) = pack2<DT>(o[0] * inv, o[1] * inv);
    if (a.lse && lane == 0)
        a.lse[(size_t)row * a.n_heads + head] =
            m == -INFINITY && l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <typename K>
cudaError_t launch(K kern, int grid, int block, size_t smem, cudaStream_t s, const AttnArgs &a,
                   int rows = -1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if constexpr (std::is_same<K, void (*)(const AttnArgs, int)>::value)
        return cudaLaunchKernelEx(&cfg, kern, a, rows);
    else
        return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int D, int DT, int RG>
cudaError_t run_main(const AttnArgs &a, cudaStream_t s) {
    constexpr size_t smem = smem_bytes<D, RG>();
    cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void *>(k_attention<D, DT, RG>), smem);
    if (e != cudaSuccess) return e;
    return launch(k_attention<D, DT, RG>, a.grid, kThreads, smem, s, a);
}

template <int D, int DT>
cudaError_t run_typed(const AttnArgs &a, int row_groups, cudaStream_t s) {
    cudaError_t e = row_groups == 1   ? run_main<D, DT, 1>(a, s)
                    : row_groups == 2 ? run_main<D, DT, 2>(a, s)
                                      : run_main<D, DT, 4>(a, s);
    if (e != cudaSuccess) return e;
    const long long rows = ((long long)a.rows * a.n_heads + 7) / 8;
    return launch(k_attention_join<D, DT>, (int)rows, 256, 0, s, a, 16 * row_groups);
}

// rows of a row tile: the smallest of 16, 32 and 64 that holds all rows of a
// key/value head
int row_groups_of(int max_rows) { return max_rows <= 16 ? 1 : max_rows <= 32 ? 2 : 4; }

typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                             const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                             const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static EncodeFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

// boxes of 64 elements and up to one page's rows, 128-byte swizzled
bool encode_rows(CUtensorMap *map, const prox_cache &c, const uint16_t *base) {
    const cuuint64_t dims[2] = {(cuuint64_t)c.head_dim,
                                (cuuint64_t)c.n_pages * c.n_kv_heads * c.page_size};
    const cuuint64_t strides[1] = {(cuuint64_t)c.head_dim * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)(c.page_size < kKT ? c.page_size : kKT)};
    const cuuint32_t ones[2] = {1, 1};
    EncodeFn fn = encode_fn();
    return fn && fn(map,
                    c.dtype == PROX_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                         : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                    2, const_cast<uint16_t *>(base), dims, strides, box, ones,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

size_t attention_part_bytes(int head_dim, int max_rows, int sms) {
    return (size_t)sms * 2 * 2 * 16 * row_groups_of(max_rows) * (head_dim + 2) * sizeof(float);
}

cudaError_t launch_attention(AttnArgs &a, const uint16_t *k_layer, int max_rows, int sms,
                             cudaStream_t s) {
    if (!encode_rows(&a.map_k, a.cache, k_layer) || !encode_rows(&a.map_v, a.cache, a.v_layer))
        return cudaErrorInvalidValue;
    a.grid = sms * 2;
    const int rg = row_groups_of(max_rows);
    const int32_t *seqs = a.seqs, *cu = a.cu_q;
    const int n = a.n;
    for (int at = 0; at < n; at += kGroup) {
        a.n = n - at < kGroup ? n - at : kGroup;
        a.seqs = seqs + at;
        a.cu_q = cu + at;
        cudaError_t e;
        if (a.cache.head_dim == 128)
            e = a.cache.dtype == PROX_BF16 ? run_typed<128, PROX_BF16>(a, rg, s)
                                           : run_typed<128, PROX_FP16>(a, rg, s);
        else
            e = a.cache.dtype == PROX_BF16 ? run_typed<64, PROX_BF16>(a, rg, s)
                                           : run_typed<64, PROX_FP16>(a, rg, s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace prox
