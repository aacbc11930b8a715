// Tree attention for more than a few rows of a key/value head: both products
// on the tensor memory's MMA (tcgen05), 128 rows a row group, one or two row
// groups a CTA, 128 keys a tile. The arithmetic and the line of tiles are those
// of k_attention.cu; what differs is where things live:
//
//   q        shared memory, K-major, 128-byte swizzle (written by the row
//            group's threads: rows are (token, head) pairs of a strided tensor)
//   k, v     a ring of shared-memory slots of 128 rows, filled by tensor-map
//            boxes; v is the second product's N-major operand as it lies
//   scores   tensor memory, one lane a row: a thread owns its row, so maxima
//            and sums need no exchange
//   probabilities over the scores they came from, in 16 bits, as the second
//            product's tensor-memory operand
//   outputs  tensor memory, fp32. They are rescaled only when a row's maximum
//            has grown by more than 2^8 since the offset in use was taken:
//            e^(x - offset) <= 2^8 loses nothing in fp32 sums.
//
// One warp loads, one thread issues the MMAs, and four warps a row group do the
// softmax. With two row groups one computes probabilities while the other's
// products run, and k and v are read once for 256 rows.
#include "attention.cuh"
#include "umma.cuh"

#include <cuda_runtime.h>

namespace prox {
namespace {

constexpr int kKT = 128;            // keys of a tile
constexpr int kMaxSlots = 10;
constexpr float kGrow = 8.f;        // log2 units a maximum may grow before outputs are rescaled

template <int D, int NWG>
struct Cfg {
    static constexpr int ROWS = 128 * NWG;
    static constexpr TileShape TS{ROWS, kKT};
    static constexpr int H = D / 64;              // 128-byte columns of a row
    static constexpr int HALF = kKT * 128;        // bytes of one of them
    static constexpr int TILE = HALF * H;         // bytes of a tile of k (or v), or of a group's q
    // slots of the ring: what fits beside q in 200 KB
    static constexpr int SLOTS = D == 128 ? (NWG == 2 ? 4 : 5) : (NWG == 2 ? 8 : 10);
    static constexpr int THREADS = 128 * NWG + 64;
    static constexpr uint32_t COLS = NWG == 2 ? 512 : 256;  // tensor-memory columns
};

struct Ctl {
    uint64_t full[kMaxSlots], empty[kMaxSlots];
    uint64_t q_ready[2], s_full[2], p_ready[2], o_full[2];
    uint64_t poison[4];             // drafted tokens whose v has an infinity or NaN
    uint32_t tmem;
};

template <int D, int NWG>
constexpr size_t smem_bytes() {
    using C = Cfg<D, NWG>;
    return 1024 + (size_t)(NWG + C::SLOTS) * C::TILE + sizeof(Line) + sizeof(Ctl);
}

// D (fp32) (+)= A (16-bit, tensor memory) x B^T
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t db, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(db), "r"(idesc), "r"(accumulate)
        : "memory");
}

// kind::f16 instruction descriptor: fp32 result, M = 128, N = n, operands of
// the given type, B N-major if b_mn
template <int DT>
__host__ __device__ constexpr uint32_t idesc_of(int n, bool b_mn) {
    return (1u << 4) | ((DT == PROX_BF16 ? 1u : 0u) << 7) | ((DT == PROX_BF16 ? 1u : 0u) << 10) |
           ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
        "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// 32 columns of this thread's lane, load and wait in one statement
__device__ __forceinline__ void tmem_get32(uint32_t taddr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
        "%28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]),
          "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]),
          "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]),
          "=r"(v[31])
        : "r"(taddr)
        : "memory");
}

// bounded wait; once one has given up, later ones do not wait at all
__device__ __forceinline__ void wait_or_give_up(uint64_t *bar, uint32_t count, const AttnArgs &a,
                                                bool &live) {
    if (live && !mbar_wait(bar, count & 1, a.wait_us)) {
        live = false;
        atomicOr(a.cache.status, PROX_CACHE_TIMEOUT);
    }
}

template <int D, int DT, int NWG>
__global__ void __launch_bounds__(Cfg<D, NWG>::THREADS, 1)
    k_attention_tc(const __grid_constant__ AttnArgs a) {
    using C = Cfg<D, NWG>;
    constexpr int ROWS = C::ROWS, H = C::H, SLOTS = C::SLOTS;
    extern __shared__ unsigned char raw[];
    unsigned char *sq = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    unsigned char *ring = sq + NWG * C::TILE;
    Line &ln = *reinterpret_cast<Line *>(ring + SLOTS * C::TILE);
    Ctl &ctl = *reinterpret_cast<Ctl *>(&ln + 1);
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const prox_cache &c = a.cache;
    const int ps = c.page_size, G = a.n_heads / c.n_kv_heads;

    if (tid == 0) {
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(&ctl.full[i], 1);
            mbar_init(&ctl.empty[i], 1);
        }
        for (int w = 0; w < NWG; ++w) {
            mbar_init(&ctl.q_ready[w], 4);
            mbar_init(&ctl.s_full[w], 1);
            mbar_init(&ctl.p_ready[w], 4);
            mbar_init(&ctl.o_full[w], 1);
        }
        mbar_fence_init();
    }
    if (wid == 4 * NWG) tmem_alloc(&ctl.tmem, C::COLS);
    pdl_wait();
    pdl_launch();
    tc_fence_before();
    build_line(ln, a, C::TS, blockIdx.x == 0);  // (its barriers cover the setup above)
    tc_fence_after();
    const uint32_t tmem = ctl.tmem;
    const uint32_t t_s = tmem, t_o = tmem + NWG * 128;  // + 128 per row group
    const long long run = run_length(ln, a.n, a.grid);
    const long long begin = min(blockIdx.x * run, ln.pre[a.n]);
    const long long end = min(begin + run, ln.pre[a.n]);
    const int per_box = min(ps, kKT), boxes = kKT / per_box;
    bool live = true;

    if (wid == 4 * NWG + 1) {
        // ------------------------------------------------------------------
        // loading warp: lane = (page of the tile, 64 elements); slot sequence
        // k0, v0, k1, v1, ...
        // ------------------------------------------------------------------
        const int pg = lane / H, half = lane % H;
        int it = 0;
        for (long long pos = begin; pos < end;) {
            const Stretch st = stretch_at(ln, a, C::TS, pos, end);
            pos += st.n_tiles;
            const int tot = ln.tot[st.b];
            const int32_t *table = c.page_table + (size_t)max(ln.seq[st.b], 0) * c.max_pages;
            auto page_of = [&](int tile) {
                const int key = tile * kKT + pg * per_box;
                return pg < boxes && key < tot ? table[key / ps] : kNone;
            };
            int page = page_of(st.tile0);
            for (int i = 0; i < st.n_tiles; ++i) {
                const int tile = st.tile0 + i;
                const int next = i + 1 < st.n_tiles ? page_of(tile + 1) : kNone;
                // a page id out of range: zeros (a box outside the map), and the mask
                const bool wanted = page != kNone, good = page >= 0 && page < c.n_pages;
                const unsigned bad = __ballot_sync(0xffffffffu, wanted && !good);
                const unsigned load = __ballot_sync(0xffffffffu, wanted);
                if (bad && lane == 0) atomicOr(c.status, PROX_CACHE_BAD_STATE);
                const int y = good ? (page * c.n_kv_heads + st.head) * ps + tile * kKT % ps
                                   : c.n_pages * c.n_kv_heads * ps;
                for (int kv = 0; kv < 2; ++kv, ++it) {
                    const int slot = it % SLOTS;
                    if (it >= SLOTS) {
                        const bool was = live;
                        if (live && !mbar_wait(&ctl.empty[slot], (it / SLOTS - 1) & 1, a.wait_us))
                            live = false;
                        if (was && !live && lane == 0) atomicOr(c.status, PROX_CACHE_TIMEOUT);
                    }
                    if (!live) break;
                    if (lane == 0)
                        mbar_arrive_expect_tx(&ctl.full[slot], __popc(load) * per_box * 128);
                    __syncwarp();
                    if (wanted)
                        asm volatile(
                            "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::"
                            "bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
                                smem_addr(ring) + slot * C::TILE + half * C::HALF + pg * per_box * 128),
                            "l"(reinterpret_cast<uint64_t>(kv ? &a.map_v : &a.map_k)),
                            "r"(half * 64), "r"(y), "r"(smem_addr(&ctl.full[slot]))
                            : "memory");
                }
                if (!live) break;
                page = next;
            }
            if (!live) break;
        }
        // after a wait that gave up: let the copies in flight land
        if (!live)
            for (int k = max(0, it - SLOTS); k < it; ++k)
                mbar_wait(&ctl.full[k % SLOTS], (k / SLOTS) & 1, 1000);
    } else if (wid == 4 * NWG) {
        // ------------------------------------------------------------------
        // the thread that issues the MMAs
        // ------------------------------------------------------------------
        if (lane == 0) {
            constexpr uint32_t qk_idesc = idesc_of<DT>(kKT, false), pv_idesc = idesc_of<DT>(D, true);
            const uint32_t qa = smem_addr(sq), ra = smem_addr(ring);
            int it = 0;
            uint32_t n_q[2] = {}, n_p[2] = {};
            auto qk = [&](int w, int slot) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    umma(t_s + w * 128,
                         sw128_desc(qa + w * C::TILE + (k / 4) * C::HALF + (k % 4) * 32, 16, 1024),
                         sw128_desc(ra + slot * C::TILE + (k / 4) * C::HALF + (k % 4) * 32, 16, 1024),
                         qk_idesc, k > 0);
                umma_commit(&ctl.s_full[w]);
            };
            for (long long pos = begin; pos < end;) {
                const Stretch st = stretch_at(ln, a, C::TS, pos, end);
                pos += st.n_tiles;
                const int groups =
                    NWG == 2 && ln.rows[st.b] * G - st.row_tile * ROWS > 128 ? 2 : 1;
                wait_or_give_up(&ctl.full[it % SLOTS], it / SLOTS, a, live);
                for (int w = 0; w < groups; ++w) {
                    wait_or_give_up(&ctl.q_ready[w], n_q[w]++, a, live);
                    tc_fence_after();
                    qk(w, it % SLOTS);
                }
                umma_commit(&ctl.empty[it % SLOTS]);
                for (int i = 0; i < st.n_tiles; ++i) {
                    const int sv = (it + 1) % SLOTS, sk = (it + 2) % SLOTS;
                    const bool more = i + 1 < st.n_tiles;
                    wait_or_give_up(&ctl.full[sv], (it + 1) / SLOTS, a, live);
                    for (int w = 0; w < groups; ++w) {
                        wait_or_give_up(&ctl.p_ready[w], n_p[w]++, a, live);
                        tc_fence_after();
#pragma unroll
                        for (int k = 0; k < kKT / 16; ++k)
                            umma_ts(t_o + w * 128, t_s + w * 128 + k * 8,
                                    sw128_desc(ra + sv * C::TILE + k * 2048, C::HALF, 1024),
                                    pv_idesc, i > 0 || k > 0);
                        if (w == groups - 1) umma_commit(&ctl.empty[sv]);
                        if (more) {
                            if (w == 0) wait_or_give_up(&ctl.full[sk], (it + 2) / SLOTS, a, live);
                            qk(w, sk);
                            if (w == groups - 1) umma_commit(&ctl.empty[sk]);
                        } else {
                            umma_commit(&ctl.o_full[w]);
                        }
                    }
                    it += 2;
                }
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------------
        // softmax: row group w, one thread a row
        // ------------------------------------------------------------------
        const int w = wid >> 2, t = tid & 127;
        const uint32_t lane_at = (uint32_t)(wid & 3) << 21;   // first tensor-memory lane << 16
        const uint32_t ts = t_s + w * 128 + lane_at, to = t_o + w * 128 + lane_at;
        const float sc = a.scale * kLog2e;
        int it = 0;
        uint32_t n_s = 0, n_o = 0;
        for (long long pos = begin; pos < end;) {
            const Stretch st = stretch_at(ln, a, C::TS, pos, end);
            const bool first = pos == begin;
            pos += st.n_tiles;
            const int len = ln.len[st.b], tot = ln.tot[st.b];
            const int n_rows = ln.rows[st.b] * G - st.row_tile * ROWS;  // of this row tile
            if (NWG == 2) named_bar_sync(2, 256);  // both groups are done with ctl.poison
            if (w * 128 >= n_rows) {
                it += 2 * st.n_tiles;
                continue;
            }
            if (w == 0 && t < 4) ctl.poison[t] = 0;
            const bool there = tid < n_rows;             // (tid = w * 128 + t)
            const bool busy = (wid * 32) < n_rows;       // the warp has rows
            const int r = st.row_tile * ROWS + tid;
            const int tok = there ? r / G : 0, head = st.head * G + (there ? r - tok * G : 0);
            const size_t row = ln.row0[st.b] + tok;
            const uint64_t *tree = a.tree ? a.tree + row * a.tree_words : nullptr;
            {
                // q: 16-byte pieces; rows behind the last one are zeros
                const uint4 *src = reinterpret_cast<const uint4 *>(a.q + row * a.q_stride + (size_t)head * D);
                unsigned char *dst = sq + w * C::TILE + t * 128;
                if (busy) {
#pragma unroll
                    for (int x = 0; x < D / 8; ++x) {
                        const uint4 v = there ? src[x] : make_uint4(0, 0, 0, 0);
                        *reinterpret_cast<uint4 *>(dst + (x >> 3) * C::HALF +
                                                   (((x & 7) ^ (t & 7)) << 4)) = v;
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.q_ready[w]);
            }
            // pages of a tile with an id out of range, one bit each (the ids of the
            // next tile are on their way while this one is worked on)
            const int32_t *table = c.page_table + (size_t)max(ln.seq[st.b], 0) * c.max_pages;
            auto peek = [&](int tile) {
                const int key = tile * kKT + lane * per_box;
                return lane < boxes && key < tot ? table[key / ps] : 0;
            };
            int page = peek(st.tile0);
            float m = -INFINITY, l = 0.f;   // offset in use (log2 units) and sum
            for (int i = 0; i < st.n_tiles; ++i, it += 2) {
                const int tile = st.tile0 + i;
                const uint32_t bad = __ballot_sync(0xffffffffu, !page_ok(c, page));
                page = i + 1 < st.n_tiles ? peek(tile + 1) : 0;
                wait_or_give_up(&ctl.s_full[w], n_s++, a, live);
                tc_fence_after();
                const bool edge = (tile + 1) * kKT > len;
                if (w == 0 && edge) {
                    // v's rows that must not meet the tensor core, one thread a
                    // key: rows behind the last key (0 * inf is not 0), and the
                    // infinities and NaN of drafted tokens, which only some rows
                    // see; those come back when the outputs are written
                    const int sv = (it + 1) % SLOTS, key = tile * kKT + t;
                    wait_or_give_up(&ctl.full[sv], (it + 1) / SLOTS, a, live);
                    unsigned char *vr = ring + sv * C::TILE + t * 128;
                    if (key >= tot) {
#pragma unroll
                        for (int x = 0; x < D / 8; ++x)
                            *reinterpret_cast<uint4 *>(vr + (x >> 3) * C::HALF + (x & 7) * 16) =
                                make_uint4(0, 0, 0, 0);
                    } else if (key >= len) {
                        bool odd = false;
                        for (int x = 0; x < D / 8; ++x) {
                            uint4 *p = reinterpret_cast<uint4 *>(vr + (x >> 3) * C::HALF + (x & 7) * 16);
                            uint4 v = *p;
                            if (non_finite2<DT>(v.x) || non_finite2<DT>(v.y) ||
                                non_finite2<DT>(v.z) || non_finite2<DT>(v.w)) {
                                odd = true;
                                v.x = finite2<DT>(v.x);
                                v.y = finite2<DT>(v.y);
                                v.z = finite2<DT>(v.z);
                                v.w = finite2<DT>(v.w);
                                *p = v;
                            }
                        }
                        if (odd)
                            atomicOr(reinterpret_cast<unsigned long long *>(
                                         &ctl.poison[(key - len) >> 6 & 3]),
                                     1ull << (key - len & 63));
                    }
                    fence_proxy_async_smem();
                }
                if (busy) {
                    const bool masked = edge || bad;
                    uint64_t seen[2] = {~0ull, ~0ull};
                    if (masked) {
#pragma unroll
                        for (int hw = 0; hw < 2; ++hw) {
                            const int w0 = tile * kKT + hw * 64;
                            uint64_t ok = low_bits(tot - w0);
                            for (int p = 0; p < boxes; ++p)
                                if (bad >> p & 1) {
                                    const int lo = p * per_box - hw * 64;
                                    ok &= ~(low_bits(lo + per_box) & ~low_bits(lo));
                                }
                            seen[hw] = there ? seen_bits(tree, a.tree_words, len, tok, w0) & ok : 0ull;
                        }
                    }
                    // the row's maximum, then its probabilities over the scores
                    float mx = -INFINITY;
#pragma unroll
                    for (int q = 0; q < kKT / 32; ++q) {
                        uint32_t s[32];
                        tmem_get32(ts + q * 32, s);
                        const uint32_t bits = (uint32_t)(seen[q >> 1] >> (q & 1) * 32);
                        if (masked) {
#pragma unroll
                            for (int x = 0; x < 32; ++x)
                                if (bits >> x & 1) mx = fmaxf(mx, __uint_as_float(s[x]));
                        } else {
#pragma unroll
                            for (int x = 0; x < 32; ++x) mx = fmaxf(mx, __uint_as_float(s[x]));
                        }
                    }
                    mx *= sc;
                    const bool grew = mx > m + kGrow || (mx > m && m == -INFINITY);
                    if (__any_sync(0xffffffffu, grew)) {
                        const float nm = fmaxf(m, mx);
                        const float f = nm > m ? ex2(m - nm) : 1.f;
                        m = nm;
                        l *= f;
                        if (i > 0) {
#pragma unroll 1
                            for (int q = 0; q < D / 32; ++q) {
                                uint32_t o[32];
                                tmem_get32(to + q * 32, o);
#pragma unroll
                                for (int x = 0; x < 32; ++x)
                                    o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
                                tmem_st16(to + q * 32, *reinterpret_cast<uint32_t(*)[16]>(&o[0]));
                                tmem_st16(to + q * 32 + 16, *reinterpret_cast<uint32_t(*)[16]>(&o[16]));
                            }
                        }
                    }
                    const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll
                    for (int q = 0; q < kKT / 32; ++q) {
                        uint32_t s[32], p[16];
                        tmem_get32(ts + q * 32, s);
                        if (masked) {
                            const uint32_t bits = (uint32_t)(seen[q >> 1] >> (q & 1) * 32);
#pragma unroll
                            for (int x = 0; x < 32; ++x)
                                if (!(bits >> x & 1)) s[x] = 0xff800000u;
                        }
#pragma unroll
                        for (int x = 0; x < 32; x += 2) {
                            const float e0 = ex2(fmaf(__uint_as_float(s[x]), sc, -mu));
                            const float e1 = ex2(fmaf(__uint_as_float(s[x + 1]), sc, -mu));
                            l += e0 + e1;
                            p[x / 2] = pack2<DT>(e0, e1);
                        }
                        tmem_st16(ts + q * 16, p);
                    }
                    tmem_st_wait();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.p_ready[w]);
            }
            // --------------------------------------------------------------
            // the rows' outputs, or a piece of them
            // --------------------------------------------------------------
            wait_or_give_up(&ctl.o_full[w], n_o++, a, live);
            tc_fence_after();
            if (busy) {
                const bool whole = st.n_tiles == st.all_tiles;
                const float inv = l == 0.f ? 0.f : whole ? 1.f / l : 1.f;
                float *part = piece(a, blockIdx.x, first, D, ROWS);
                const uint64_t any = ctl.poison[0] | ctl.poison[1] | ctl.poison[2] | ctl.poison[3];
#pragma unroll 1
                for (int q = 0; q < D / 32; ++q) {
                    uint32_t ob[32];
                    tmem_get32(to + q * 32, ob);
                    float o[32];
#pragma unroll
                    for (int x = 0; x < 32; ++x) o[x] = __uint_as_float(ob[x]) * inv;
                    if (any && there) {
                        for (int k = 0; k < 4; ++k) {
                            uint64_t bits = ctl.poison[k];
                            bits &= tree ? (k < a.tree_words ? tree[k] : 0ull)
                                         : low_bits(tok + 1 - k * 64);
                            for (; bits; bits &= bits - 1) {
                                const int key = len + k * 64 + __ffsll((long long)bits) - 1;
                                const int page =
                                    c.page_table[(size_t)ln.seq[st.b] * c.max_pages + key / ps];
                                if (!page_ok(c, page)) continue;  // (cannot be: its box was read)
                                const uint32_t *v = reinterpret_cast<const uint32_t *>(
                                    a.v_layer +
                                    (((size_t)page * c.n_kv_heads + st.head) * ps + key % ps) * D + q * 32);
#pragma unroll
                                for (int x = 0; x < 32; x += 2) {
                                    const uint32_t vv = v[x / 2];
                                    if (!non_finite2<DT>(vv)) continue;
                                    const float2 f = unpack2<DT>(vv);
                                    if (!isfinite(f.x)) o[x] += f.x;
                                    if (!isfinite(f.y)) o[x + 1] += f.y;
                                }
                            }
                        }
                    }
                    if (!whole) {
#pragma unroll
                        for (int x = 0; x < 32; x += 4)
                            reinterpret_cast<float4 *>(part)[(size_t)(q * 8 + x / 4) * ROWS + tid] =
                                make_float4(o[x], o[x + 1], o[x + 2], o[x + 3]);
                    } else if (there) {
                        uint4 *op = reinterpret_cast<uint4 *>(a.out + row * a.out_stride +
                                                              (size_t)head * D + q * 32);
#pragma unroll
                        for (int x = 0; x < 32; x += 8)
                            op[x / 8] = make_uint4(pack2<DT>(o[x], o[x + 1]), pack2<DT>(o[x + 2], o[x + 3]),
                                                   pack2<DT>(o[x + 4], o[x + 5]),
                                                   pack2<DT>(o[x + 6], o[x + 7]));
                    }
                }
                if (!whole) {
                    part[ROWS * D + tid] = m;
                    part[ROWS * (D + 1) + tid] = l;
                } else if (there && a.lse) {
                    a.lse[row * a.n_heads + head] =
                        m == -INFINITY && l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
                }
            }
            tc_fence_before();  // outputs are read: the next stretch may overwrite them
        }
    }
    __syncthreads();
    if (wid == 4 * NWG) tmem_free(tmem, C::COLS);
}

template <int D, int DT, int NWG>
cudaError_t run(const AttnArgs &a, cudaStream_t s) {
    constexpr size_t smem = smem_bytes<D, NWG>();
    static_assert(smem <= 227 * 1024, "shared memory of one CTA");
    auto kern = k_attention_tc<D, DT, NWG>;
    cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void *>(kern), smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(a.grid), dim3(Cfg<D, NWG>::THREADS), smem, s, a);
}

}  // namespace

cudaError_t launch_attention_tc(const AttnArgs &a, int row_groups, cudaStream_t s) {
    const bool two = row_groups == 2, bf = a.cache.dtype == PROX_BF16;
    if (a.cache.head_dim == 128)
        return bf ? two ? run<128, PROX_BF16, 2>(a, s) : run<128, PROX_BF16, 1>(a, s)
                  : two ? run<128, PROX_FP16, 2>(a, s) : run<128, PROX_FP16, 1>(a, s);
    return bf ? two ? run<64, PROX_BF16, 2>(a, s) : run<64, PROX_BF16, 1>(a, s)
              : two ? run<64, PROX_FP16, 2>(a, s) : run<64, PROX_FP16, 1>(a, s);
}

}  // namespace prox
