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
// with mma.sync m16n8k16 (bf16 or fp16, fp32 sums) on tiles of 16 or 32 rows:
// with so few rows the tensor pipes keep up with the memory, and a warp's
// registers carry a tile of scores straight into the second product. More
// rows take the kernel of k_attention_tc.cu; plan_of has the rule.
//
// Measured on the device, back to back: one token of 32 heads over 1,021 tokens
// 9.6 us, 8 tokens over 16,383 (67 MB of k and v) 26.5 us, 2.5 TB/s. Of the latter
// 6 us pass before the first tile is there (lengths, line, page ids, tiles: reads
// that wait for one another) and 3.4 us go to the join; the tiles between them
// come at 4 TB/s.
#include "attention.cuh"

#include <cuda_runtime.h>
#include <cstdint>
#include <type_traits>

namespace prox {
namespace {

constexpr int kWarps = 4;           // computing warps
constexpr int kThreads = 32 * kWarps + 32;
constexpr int kMaxStages = 8;
constexpr int kMaxGrid = 512;        // CTAs of a main kernel

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

// (control data lies behind the line in shared memory)
static_assert(sizeof(Line) % 16 == 0, "barriers are 8-byte aligned");

struct Ctl {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t poison;              // drafted keys of the tile whose v is not finite
    uint32_t dead;                // a wait has given up
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
        ctl.dead = 0;
        mbar_fence_init();
    }
    pdl_wait();
    pdl_launch();
    build_line(ln, a, ROWS, blockIdx.x == 0);  // (its barriers cover the mbarriers too)
    const int run = run_length(ln, a.n, a.grid), total = ln.pre[a.n];
    if (blockIdx.x > (total - 1) / run || total == 0) return;
    const int begin = blockIdx.x * run, end = begin + min(run, total - begin);
    const int per_box = min(ps, kKT);           // rows of a box
    const int boxes = kKT / per_box;            // pages of a tile

    if (wid == kWarps) {
        // ------------------------------------------------------------------
        // loading warp: lane = (page of the tile, k or v, 64 elements)
        // ------------------------------------------------------------------
        constexpr int H = D / 64;
        const uint64_t policy = l2_evict_first();
        const int pg = lane / (2 * H), kv = lane / H & 1, half = lane % H;
        bool live = true;
        int it = 0;
        for (int pos = begin; pos < end;) {
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
                if (!__all_sync(0xffffffffu, it < NST || mbar_spin(&ctl.empty[slot], (it / NST - 1) & 1,
                                                                   a.wait_us, &ctl.dead))) {
                    live = false;
                    ctl.dead = 1;
                    if (lane == 0) atomicOr(c.status, PROX_CACHE_TIMEOUT);
                    break;
                }
                // a page id out of range: zeros (a box outside the map), and the mask
                const bool wanted = page != kNone, good = page >= 0 && page < c.n_pages;
                const unsigned bad = __ballot_sync(0xffffffffu, wanted && !good);
                const unsigned load = __ballot_sync(0xffffffffu, wanted);
                const bool skip = blockIdx.x == 0 && it == a.debug_skip;
                if (lane == 0 && !skip) {
                    uint32_t pages = 0;
                    for (int p = 0; p < boxes; ++p) pages |= (bad >> (p * 2 * H) & 1u) << p;
                    if (pages) atomicOr(c.status, PROX_CACHE_BAD_STATE);
                    ctl.bad[slot] = pages;
                    mbar_arrive_expect_tx(&ctl.full[slot], __popc(load) * per_box * 128);
                }
                __syncwarp();
                if (wanted && !skip) {
                    const int y = good ? (page * c.n_kv_heads + st.head) * ps + tile * kKT % ps
                                       : c.n_pages * c.n_kv_heads * ps;
                    box_g2s(smem_addr(sm) + slot * 2 * C::TILE + kv * C::TILE + half * C::HALF +
                                pg * per_box * 128,
                            kv ? &a.map_v : &a.map_k, half * 64, y, &ctl.full[slot], policy);
                }
                page = next;
            }
            if (!live) break;
        }
        // no copy is in flight when the CTA ends, not behind a wait that gave up either
        // (whatever its bound was)
        for (int k = max(0, it - NST); k < it; ++k)
            if (blockIdx.x > 0 || k != a.debug_skip)
                mbar_spin(&ctl.full[k % NST], (k / NST) & 1, kDefaultWaitUs);
        return;
    }

    // ----------------------------------------------------------------------
    // computing warps
    // ----------------------------------------------------------------------
    const int rg = wid % RG, kg = wid / RG, g = lane >> 2, tg = lane & 3;
    const float sc = a.scale_log2;
    bool live = true;
    int it = 0;
    for (int pos = begin; pos < end;) {
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
        bool big = false;  // a row of the warp has an offset beyond kRoundFirst

        for (int i = 0; i < st.n_tiles; ++i, ++it) {
            const int tile = st.tile0 + i, slot = it % NST;
            if (live && !mbar_spin(&ctl.full[slot], (it / NST) & 1, a.wait_us, &ctl.dead)) {
                live = false;
                ctl.dead = 1;
                if (lane == 0) atomicOr(c.status, PROX_CACHE_TIMEOUT);
            }
            __syncwarp();  // (lanes may have seen the phase end at different tries)
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
                big = __any_sync(0xffffffffu, fmaxf(fabsf(mu[0]), fabsf(mu[1])) >= kRoundFirst);
#pragma unroll
                for (int d = 0; d < DB; ++d) {
                    o[d][0] *= r[0];
                    o[d][1] *= r[0];
                    o[d][2] *= r[1];
                    o[d][3] *= r[1];
                }
            }
            if (big)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int x = 0; x < 4; ++x) s[nb][x] = __fmul_rn(s[nb][x], sc);
            const float by = big ? 1.f : sc;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    s[nb][x] = ex2(fmaf(s[nb][x], by, -mu[x >> 1]));
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
            // (a slot that was not waited for may be under way: it is not given back)
            if (lane == 0 && live) mbar_arrive(&ctl.empty[slot]);
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
                float *part = piece(a, blockIdx.x, first, D, ROWS), *pm = part + ROWS * D;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = rg * 16 + g + 8 * e;
#pragma unroll
                    for (int d = 0; d < DB; ++d)
                        *reinterpret_cast<float2 *>(
                            part + ((size_t)(d * 2 + (tg >> 1)) * ROWS + r) * 4 + (tg & 1) * 2) =
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

// the cuts that join a unit: inside one, and the first there
struct Cuts {
    uint16_t at[kMaxGrid];
    int warp[8];
};
__device__ int joining_cuts(const Line &ln, const AttnArgs &a, int ROWS, Cuts &c) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int run = run_length(ln, a.n, a.grid), total = ln.pre[a.n];
    const int cuts = total ? (total - 1) / run : 0;
    int count = 0;
    for (int b = 0; b < cuts; b += 256) {
        const int j = b + threadIdx.x, cut = (j + 1) * run;
        bool joins = false;
        if (j < cuts) {
            const Stretch st = stretch_at(ln, a, ROWS, cut, total);
            joins = st.tile0 > 0 && j * run <= cut - st.tile0;
        }
        const unsigned who = __ballot_sync(0xffffffffu, joins);
        __syncthreads();
        if (lane == 0) c.warp[wid] = __popc(who);
        __syncthreads();
        int at = count;
        for (int w = 0; w < 8; ++w) {
            if (w < wid) at += c.warp[w];
            count += c.warp[w];
        }
        if (joins) c.at[at + __popc(who & ((1u << lane) - 1))] = (uint16_t)j;
    }
    __syncthreads();
    return count;
}

// Joins the pieces of units that were cut. A unit is cut where a CTA's run ends
// inside it, so the cuts are numbered by the CTAs, and a unit is joined by the
// first cut in it. The CTAs share out steps of 32 rows and CC columns: lanes are
// rows (a piece is read in runs of 512 bytes), the pieces are dealt out to the
// warps, whose sums meet in shared memory in a fixed order. All reads of BATCH
// pieces a warp are in flight at once. What has to be joined is worked out before
// the wait for the main kernel: on an SM whose CTAs of that kernel have ended (beside
// them its registers leave no room). Notes that its CTAs left in the workspace instead
// cost two more reads behind it: 11.4 against 9.8 us for one token over 1,021.
template <int D, int DT, int CC, int BATCH>
__global__ void __launch_bounds__(256, BATCH > 2 ? 1 : 2)
    k_attention_join(const __grid_constant__ AttnArgs a, int ROWS) {
    __shared__ Line ln;
    __shared__ float s_o[8][CC][32], s_m[8][32], s_l[8][32];
    __shared__ Cuts cuts;
    // The line depends on the call's inputs alone, which were there before the
    // main kernel let this one start; its pieces come after the wait.
    build_line(ln, a, ROWS, false);
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int G = a.n_heads / a.cache.n_kv_heads;
    const int row_groups = (ROWS + 31) / 32, per_cut = row_groups * (D / CC);
    const int run = run_length(ln, a.n, a.grid), total = ln.pre[a.n];
    const int count = joining_cuts(ln, a, ROWS, cuts);
    const int items = count * per_cut;
    bool waited = false;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int j = cuts.at[item / per_cut], rest = item % per_cut, cut = (j + 1) * run;
        const Stretch st = stretch_at(ln, a, ROWS, cut, total);
        const int u0 = cut - st.tile0, u1 = u0 + st.all_tiles;
        const int cc = rest % (D / CC), row0 = st.row_tile * ROWS + rest / (D / CC) * 32;
        const int n_rows = ln.rows[st.b] * G;
        if (row0 >= n_rows) continue;
        const int r = row0 + lane, rr = r % ROWS;  // (rows behind the last: any row's place)
        const int c1 = (u1 - 1) / run;
        if (!waited) pdl_wait();
        waited = true;
        // pieces j .. c1, this warp's ones under a running maximum
        float M = -INFINITY, l = 0.f;
        float4 o[CC / 4] = {};
        for (int c = j + wid; c <= c1; c += 8 * BATCH) {
            float4 v[BATCH][CC / 4];
            float pm[BATCH], pl[BATCH];
#pragma unroll
            for (int u = 0; u < BATCH; ++u) {
                const int k = c + 8 * u;
                pm[u] = -INFINITY;
                pl[u] = 0.f;
                if (k <= c1) {
                    const float *p = piece(a, k, k * run >= u0, D, ROWS);
                    const float4 *x = reinterpret_cast<const float4 *>(p) + cc * (CC / 4) * ROWS + rr;
#pragma unroll
                    for (int y = 0; y < CC / 4; ++y) v[u][y] = __ldcg(x + y * ROWS);
                    pm[u] = __ldcg(p + ROWS * D + rr);
                    pl[u] = __ldcg(p + ROWS * (D + 1) + rr);
                }
            }
            float nm = M;
#pragma unroll
            for (int u = 0; u < BATCH; ++u) nm = fmaxf(nm, pm[u]);
            const float mu = nm == -INFINITY ? 0.f : nm, f0 = ex2(M - mu);
            M = nm;
            l *= f0;
#pragma unroll
            for (int y = 0; y < CC / 4; ++y) {
                o[y].x *= f0;
                o[y].y *= f0;
                o[y].z *= f0;
                o[y].w *= f0;
            }
#pragma unroll
            for (int u = 0; u < BATCH; ++u) {
                if (c + 8 * u > c1) continue;
                const float f = ex2(pm[u] - mu);
                l = fmaf(f, pl[u], l);
#pragma unroll
                for (int y = 0; y < CC / 4; ++y) {
                    o[y].x = fmaf(f, v[u][y].x, o[y].x);
                    o[y].y = fmaf(f, v[u][y].y, o[y].y);
                    o[y].z = fmaf(f, v[u][y].z, o[y].z);
                    o[y].w = fmaf(f, v[u][y].w, o[y].w);
                }
            }
        }
        const int parts = min(c1 - j + 1, 8);
        __syncthreads();  // the last step's sums are read
        if (wid < parts) {
            s_m[wid][lane] = M;
            s_l[wid][lane] = l;
#pragma unroll
            for (int k = 0; k < CC / 4; ++k) {
                s_o[wid][4 * k][lane] = o[k].x;
                s_o[wid][4 * k + 1][lane] = o[k].y;
                s_o[wid][4 * k + 2][lane] = o[k].z;
                s_o[wid][4 * k + 3][lane] = o[k].w;
            }
        }
        __syncthreads();
        M = -INFINITY;
        for (int w = 0; w < parts; ++w) M = fmaxf(M, s_m[w][lane]);
        const float top = M == -INFINITY ? 0.f : M;
        constexpr int V = CC / 8;  // columns a warp
        float y[V] = {};
        l = 0.f;
        for (int w = 0; w < parts; ++w) {
            const float f = ex2(s_m[w][lane] - top);
            l += f * s_l[w][lane];
#pragma unroll
            for (int k = 0; k < V; ++k) y[k] = fmaf(f, s_o[w][wid * V + k][lane], y[k]);
        }
        if (r < n_rows) {
            const int t = r / G, hq = st.head * G + r - t * G;
            const size_t row = ln.row0[st.b] + t;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            uint32_t *op = reinterpret_cast<uint32_t *>(a.out + row * a.out_stride + (size_t)hq * D +
                                                        cc * CC + wid * V);
#pragma unroll
            for (int k = 0; k < V; k += 2) op[k / 2] = pack2<DT>(y[k] * inv, y[k + 1] * inv);
            if (a.lse && cc == 0 && wid == 0)
                a.lse[row * a.n_heads + hq] =
                    M == -INFINITY && l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2;
        }
    }
    // every CTA waits before it ends: what follows this kernel in the stream
    // counts on the main kernel being done
    if (!waited) pdl_wait();
    pdl_launch();
}

// The same for many units of few pieces each (a batch): a step is 32 rows with
// all columns, a warp has 1/8 of them and goes through the pieces one after
// another, three at a time in flight. No sums cross warps.
template <int D, int DT>
__global__ void __launch_bounds__(256, 3)
    k_attention_join_few(const __grid_constant__ AttnArgs a, int ROWS) {
    __shared__ Line ln;
    __shared__ Cuts cuts;
    build_line(ln, a, ROWS, false);
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int G = a.n_heads / a.cache.n_kv_heads;
    const int row_groups = (ROWS + 31) / 32;
    const int run = run_length(ln, a.n, a.grid), total = ln.pre[a.n];
    const int items = joining_cuts(ln, a, ROWS, cuts) * row_groups;
    pdl_wait();
    pdl_launch();
    constexpr int V = D / 32, BATCH = 3;  // float4 columns of a warp
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const int j = cuts.at[item / row_groups], cut = (j + 1) * run;
        const Stretch st = stretch_at(ln, a, ROWS, cut, total);
        const int u0 = cut - st.tile0, c1 = (u0 + st.all_tiles - 1) / run;
        const int row0 = st.row_tile * ROWS + item % row_groups * 32, n_rows = ln.rows[st.b] * G;
        if (row0 >= n_rows) continue;
        const int r = row0 + lane, rr = r % ROWS;  // (rows behind the last: any row's place)
        float M = -INFINITY, l = 0.f;
        float4 o[V] = {};
        for (int c = j; c <= c1; c += BATCH) {
            float4 v[BATCH][V];
            float pm[BATCH], pl[BATCH];
#pragma unroll
            for (int u = 0; u < BATCH; ++u) {
                pm[u] = -INFINITY;
                pl[u] = 0.f;
                if (c + u <= c1) {
                    const float *p = piece(a, c + u, (c + u) * run >= u0, D, ROWS);
                    const float4 *x = reinterpret_cast<const float4 *>(p) + wid * V * ROWS + rr;
#pragma unroll
                    for (int y = 0; y < V; ++y) v[u][y] = __ldcg(x + y * ROWS);
                    pm[u] = __ldcg(p + ROWS * D + rr);
                    pl[u] = __ldcg(p + ROWS * (D + 1) + rr);
                }
            }
            float nm = M;
#pragma unroll
            for (int u = 0; u < BATCH; ++u) nm = fmaxf(nm, pm[u]);
            const float mu = nm == -INFINITY ? 0.f : nm, f0 = ex2(M - mu);
            M = nm;
            l *= f0;
#pragma unroll
            for (int y = 0; y < V; ++y) {
                o[y].x *= f0;
                o[y].y *= f0;
                o[y].z *= f0;
                o[y].w *= f0;
            }
#pragma unroll
            for (int u = 0; u < BATCH; ++u) {
                if (c + u > c1) continue;
                const float f = ex2(pm[u] - mu);
                l = fmaf(f, pl[u], l);
#pragma unroll
                for (int y = 0; y < V; ++y) {
                    o[y].x = fmaf(f, v[u][y].x, o[y].x);
                    o[y].y = fmaf(f, v[u][y].y, o[y].y);
                    o[y].z = fmaf(f, v[u][y].z, o[y].z);
                    o[y].w = fmaf(f, v[u][y].w, o[y].w);
                }
            }
        }
        if (r >= n_rows) continue;
        const int t = r / G, hq = st.head * G + r - t * G;
        const size_t row = ln.row0[st.b] + t;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint4 *op = reinterpret_cast<uint4 *>(a.out + row * a.out_stride + (size_t)hq * D + wid * V * 4);
#pragma unroll
        for (int y = 0; y < V; y += 2)
            op[y / 2] = make_uint4(pack2<DT>(o[y].x * inv, o[y].y * inv), pack2<DT>(o[y].z * inv, o[y].w * inv),
                                   pack2<DT>(o[y + 1].x * inv, o[y + 1].y * inv),
                                   pack2<DT>(o[y + 1].z * inv, o[y + 1].w * inv));
        if (a.lse && wid == 0)
            a.lse[row * a.n_heads + hq] =
                M == -INFINITY && l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2;
    }
}

template <typename... P, typename... A>
cudaError_t launch(void (*kern)(P...), int grid, int block, size_t smem, cudaStream_t s,
                   const A &...args) {
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
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int D, int DT, int RG>
cudaError_t run_main(const AttnArgs &a, cudaStream_t s) {
    constexpr size_t smem = smem_bytes<D, RG>();
    cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void *>(k_attention<D, DT, RG>), smem);
    if (e != cudaSuccess) return e;
    return launch(k_attention<D, DT, RG>, a.grid, kThreads, smem, s, a);
}

// How a call runs, by the rows of a key/value head (drafted tokens x heads that
// share it) and the number of heads over all sequences: row tiles of 16 or 32 rows
// on mma.sync, of 128 or 256 rows on the tensor memory's MMA. Measured (us, head
// dim 128, 8 key/value heads of 4 heads, 64-token pages; mma.sync | tcgen05):
//                            4 rows      16 rows     32 rows     48 rows
//   1 sequence of 1,021     9.6 | 14.0   9.6 | 15.6  10.3 | 16.1   - | 16.5
//   1 sequence of 16,383   20.7 | 27.1  23.4 | 30.3  26.4 | 31.3   - | 32.1
//   24 sequences of 3,000  58.5 | 62.9  59.7 | 64.4  75.9 | 65.6   - | 69.2
// The same holds with 2 key/value heads (one of 16,383: 14.0 | 16.7 with 4 rows, 17.8
// | 22.4 with 32; 24 of 3,000: 23.3 | 32.0 and 28.7 | 35.2, above the rule's border
// only in the last), with dim 64 (15.7 | 20.0, 19.0 | 20.5; 42.5 | 44.7, 54.0 | 44.9)
// and with 16-token pages (20.5 | 26.0, 25.6 | 30.6; 58.2 | 63.9, 72.4 | 66.8).
// Tiles of 128 | 256 rows (the former have two CTAs an SM, but read k and v again for
// each 128 rows), by dim and key/value heads:
//                                      128, 8         64, 8         128, 2
//   1 of 16,383, 48 rows            31.5 | 34.0   20.0 | 28.1   23.2 | 23.3
//   24 of 3,000, 128 rows           75.6 | 93.2   54.5 | 75.3   38.4 | 32.7
//   1 of 32,749, 256 rows           62.3 | 59.6   45.9 | 50.4   30.9 | 34.0
//   16 of 8,000, 192 rows          192.9 | 158.2 132.8 | 138.9  67.9 | 65.0
// More than 128 rows take 256 for the batches of dim 128; dim 64 would gain 4 to 9%
// by 128.
struct Plan {
    int rows, grid_per_sm;
    bool tc;
};
Plan plan_of(int max_rows, long long heads, int sms) {
    if (max_rows <= 16) return {16, 2, false};
    if (max_rows <= 32 && heads * 2 < sms) return {32, 2, false};
    if (max_rows <= 128) return {128, 2, true};
    return {256, 1, true};
}

template <int D, int DT>
cudaError_t run_typed(const AttnArgs &a, const Plan &p, int max_rows, cudaStream_t s) {
    cudaError_t e = p.tc              ? launch_attention_tc(a, p.rows / 128, s)
                    : p.rows == 16 ? run_main<D, DT, 1>(a, s)
                                      : run_main<D, DT, 2>(a, s);
    if (e != cudaSuccess) return e;
    // One long sequence is cut into many pieces a unit, a batch into few. The
    // former's steps want every piece's read in flight at once if the SMs have
    // one step each at most, and two CTAs an SM otherwise. Whole calls (us; few |
    // <16, 6> | <32, 2>; dim 128, 8 key/value heads):
    //   1 of 1,021, 4 rows       20.0 |  9.6 | 10.9   16 of 4,000, 4 rows   53.5 |  73.3 | 55.6
    //   1 of 16,383, 4 rows      47.7 | 20.8 | 23.0   32 of 2,000, 4 rows   53.9 |  87.8 | 60.2
    //   1 of 16,383, 32 rows     56.6 | 26.4 | 29.6   32 of 2,000, 32 rows  61.9 | 120.4 | 82.3
    //   4 of 4,000, 16 rows      27.6 | 24.4 | 21.1   1 of 8,000, 128 rows  45.8 |  29.4 | 28.4
    //   8 of 4,000, 4 rows       34.8 | 42.0 | 31.1   1 of 32,749, 256 rows 76.7 |  68.1 | 59.4
    // (4 of 8,000 with 256 rows, 32 units: 61.7 | 91.8 | 68.0, where the rule's border
    // lies too high.)
    const long long units = (long long)a.n * a.cache.n_kv_heads * ((max_rows + p.rows - 1) / p.rows);
    const long long steps = min((long long)a.grid - 1, units) * ((p.rows + 31) / 32);  // of 32 rows
    const int sms = a.grid / p.grid_per_sm;
    if (units * 4 >= a.grid)
        return launch(k_attention_join_few<D, DT>, (int)min(steps, 4LL * sms), 256, 0, s, a, p.rows);
    if (steps * (D / 16) <= sms)
        return launch(k_attention_join<D, DT, 16, 6>, (int)steps * (D / 16), 256, 0, s, a, p.rows);
    return launch(k_attention_join<D, DT, 32, 2>, (int)min(steps * (D / 32), 4LL * sms), 256, 0, s, a,
                  p.rows);
}

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

// tiles that one sequence can have at most, in the smallest row tiles
static long long tiles_of_one(const prox_cache &c, int max_rows) {
    const int rows = max_rows <= 128 ? 128 : 256;  // (fewer rows are one tile of any kind)
    return (long long)c.n_kv_heads * ((max_rows + rows - 1) / rows) *
           ((long long)c.max_pages * c.page_size / kKT + 1);
}

bool attention_fits(const prox_cache &c, int max_rows) { return tiles_of_one(c, max_rows) < 1ll << 31; }

size_t attention_part_bytes(int head_dim, int max_rows, int sms) {
    // (for any number of heads: many take the larger row tile)
    const Plan p = plan_of(max_rows, 1 << 30, sms);
    const size_t grid = min(sms * p.grid_per_sm, kMaxGrid);
    return grid * 2 * piece_floats(head_dim, p.rows) * sizeof(float);
}

cudaError_t launch_attention(AttnArgs &a, const uint16_t *k_layer, int max_rows, int sms,
                             cudaStream_t s) {
    const Plan p = plan_of(max_rows, (long long)min(a.n, kGroup) * a.cache.n_kv_heads, sms);
    if (!encode_rows(&a.map_k, a.cache, k_layer) || !encode_rows(&a.map_v, a.cache, a.v_layer))
        return cudaErrorInvalidValue;
    a.grid = min(sms * p.grid_per_sm, kMaxGrid);
    const int32_t *seqs = a.seqs, *cu = a.cu_q;
    const int n = a.n;
    // sequences of a launch: at most kGroup, and fewer than 2^31 tiles
    const long long most = tiles_of_one(a.cache, max_rows);
    const int group = (int)min((long long)kGroup, 0x7fffffffLL / most);
    for (int at = 0; at < n; at += group) {
        a.n = n - at < group ? n - at : group;
        a.seqs = seqs + at;
        a.cu_q = cu + at;
        cudaError_t e;
        if (a.cache.head_dim == 128)
            e = a.cache.dtype == PROX_BF16 ? run_typed<128, PROX_BF16>(a, p, max_rows, s)
                                           : run_typed<128, PROX_FP16>(a, p, max_rows, s);
        else
            e = a.cache.dtype == PROX_BF16 ? run_typed<64, PROX_BF16>(a, p, max_rows, s)
                                           : run_typed<64, PROX_FP16>(a, p, max_rows, s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace prox
