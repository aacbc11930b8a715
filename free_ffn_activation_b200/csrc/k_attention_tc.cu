// Tree attention for more than a few rows of a key/value head: both products
// on the tensor memory's MMA (tcgen05), 128 rows a row group, one or two row
// groups a CTA. The arithmetic and the line of tiles are those of
// k_attention.cu; what differs is where things live:
//
//   q        shared memory, K-major, 128-byte swizzle (written by the row
//            group's threads: rows are (token, head) pairs of a strided tensor)
//   k, v     a ring of shared-memory slots of 64 rows, filled by tensor-map
//            boxes; v is the second product's N-major operand as it lies
//   scores   tensor memory, two buffers of 64 columns a row group, one lane a
//            row: a thread owns its row, so maxima and sums need no exchange
//   probabilities over the scores they came from, in 16 bits, as the second
//            product's tensor-memory operand
//   outputs  tensor memory, fp32. They are rescaled only when a row's maximum
//            has grown by more than 2^8 since the offset in use was taken:
//            e^(x - offset) <= 2^8 loses nothing in fp32 sums.
//
// One warp loads, one thread a row group issues its MMAs, and four warps a row
// group do the softmax, a row a thread with up to 168 registers: a tile's scores
// stay in registers from the maximum to the probabilities, half of the next
// tile's are fetched meanwhile, and their product runs one tile ahead. k and v
// are read once for 256 rows.
//
// What bounds it: a tile of 64 keys and 256 rows takes 1,850 to 2,150 cycles, its
// MMAs 1,200 and its exponentials 1,024 of a scheduler's special-function unit; the
// rest is the softmax warps' own chain (fetch 100, maximum 350 to 450, two waits of
// 170), two warps a scheduler. Measured: 64 tokens of 32 heads over 32,749 tokens
// 62 us (550 TFLOP/s; 6 us before the first scores, 7 us of joining, 28 tiles a CTA
// 29 us; the other 20 are not accounted for by these: the mean SM is active for 71% of
// the time, the slowest for 89%), 16 sequences with 40 to 64 tokens over 8,000 to 32,000 420 us in short runs
// (725 TFLOP/s), 470 to 500 us by GPU in long ones at 1000 W, where the clock falls
// to 1.6 GHz.
#include "attention.cuh"
#include "umma.cuh"

#include <cuda_runtime.h>

namespace prox {
namespace {

constexpr int kMaxSlots = 20;
constexpr float kGrow = 8.f;        // log2 units a maximum may grow before outputs are rescaled

template <int D, int NWG>
struct Cfg {
    static constexpr int ROWS = 128 * NWG;
    static constexpr int H = D / 64;              // 128-byte columns of a row
    static constexpr int HALF = kKT * 128;        // bytes of one of them, of a tile of k (or v)
    static constexpr int TILE = HALF * H;         // bytes of a tile of k (or v)
    static constexpr int QHALF = 128 * 128, QTILE = QHALF * H;  // the same of a group's q
    // one CTA of two row groups fills an SM's tensor memory; of one row group,
    // two CTAs do
    static constexpr int PER_SM = 3 - NWG;
    // slots of the ring: what fits beside q
    static constexpr int ROOM = (NWG == 2 ? 210 : 102) * 1024;
    static constexpr int SLOTS =
        (ROOM - NWG * QTILE) / TILE < kMaxSlots ? (ROOM - NWG * QTILE) / TILE : kMaxSlots;
    static constexpr int SOFT = 128 * NWG;        // softmax threads
    static constexpr int THREADS = SOFT + 32 * NWG + 32;
    static constexpr uint32_t COLS = NWG == 2 ? 512 : 256;  // tensor-memory columns
};

// (control data lies behind the line in shared memory)
static_assert(sizeof(Line) % 16 == 0, "barriers are 8-byte aligned");

struct Ctl {
    uint64_t full[kMaxSlots], empty[kMaxSlots];
    // per row group: q written; scores there and probabilities there (two
    // buffers); the second products of a stretch done but for its last tile's, and all
    uint64_t q_ready[2], s_full[2][2], p_ready[2][2], o_done[2], o_full[2];
    uint64_t poison[2][4];          // drafted tokens whose v has an infinity or NaN (by stretch parity)
    uint64_t drained[2];            // all of a row group's MMAs are done
    uint32_t tmem, dead;            // a wait has given up
};

template <int D, int NWG>
constexpr size_t smem_bytes() {
    using C = Cfg<D, NWG>;
    return 1024 + (size_t)NWG * C::QTILE + (size_t)C::SLOTS * C::TILE + sizeof(Line) + sizeof(Ctl);
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

// 32 columns of this thread's lane on their way; tmem_take32 makes them usable
__device__ __forceinline__ void tmem_ask32(uint32_t taddr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
        "%28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]),
          "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]),
          "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]),
          "=r"(v[31])
        : "r"(taddr)
        : "memory");
}
// (the registers go through the wait, so that no use of them can precede it)
__device__ __forceinline__ void tmem_take32(uint32_t (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]),
                   "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]),
                   "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]), "+r"(v[17]),
                   "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]),
                   "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]),
                   "+r"(v[30]), "+r"(v[31])
                 :
                 : "memory");
}

// two fp32 operations an instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// one thread of the warp, the same one each time
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(p));
    return p != 0;
}
// a value that is the same in all lanes, in a form that says so
template <typename T>
__device__ __forceinline__ T uniform(T x) {
    return __shfl_sync(0xffffffffu, x, 0);
}

// The queries into L2, a few lines a thread, by all CTAs together: where each
// CTA's rows are is known only after the line, and its reads would then stand
// behind the first stages of keys and values of all CTAs (64 drafted tokens of 32
// heads over 32,749 tokens: 62.1 -> 61.5 us when it was added).
__device__ __forceinline__ void prefetch_queries(const AttnArgs &a, int D) {
    const unsigned per_row = a.n_heads * (D / 64);  // lines of 128 bytes
    const unsigned step = gridDim.x * blockDim.x;
    const unsigned lines = (unsigned)min((long long)a.rows * per_row, 4ll * step);
    for (unsigned i = ((threadIdx.x >> 5) * gridDim.x + blockIdx.x) * 32 + (threadIdx.x & 31); i < lines;
         i += step) {
        const unsigned row = i / per_row;
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.q + row * a.q_stride + (i - row * per_row) * 64));
    }
}

// bounded wait of a whole warp; once one has given up, later ones do not wait at
// all. Lanes may see the phase end at different tries, and what follows (named
// barriers, tensor-memory loads) wants the warp together again.
__device__ __forceinline__ void wait_or_give_up(uint64_t *bar, uint32_t count, const AttnArgs &a,
                                                Ctl &ctl, bool &live) {
    if (live && !mbar_spin(bar, count & 1, a.wait_us, &ctl.dead)) {
        live = false;
        ctl.dead = 1;
        atomicOr(a.cache.status, PROX_CACHE_TIMEOUT);
    }
    __syncwarp();
}

// e^(score - offset) of one query row and one key, for the drafted tokens whose v
// the tensor core must not see (offset in units of log 2). q is a row group's tile in
// shared memory (a row's output may lie where the row was read from), t the row. Rare,
// so kept out of the kernel's registers.
template <int D, int DT>
__device__ __noinline__ float draft_weight(const unsigned char *q, int t, const uint16_t *k, float sc,
                                           float offset) {
    float x = 0.f;
#pragma unroll 1
    for (int d = 0; d < D; d += 2) {
        const int y = d >> 3;  // 16-byte piece
        const float2 a = unpack2<DT>(*reinterpret_cast<const uint32_t *>(
                         q + t * 128 + (y >> 3) * (128 * 128) + (((y & 7) ^ (t & 7)) << 4) + (d & 7) * 2)),
                     b = unpack2<DT>(*reinterpret_cast<const uint32_t *>(k + d));
        x = fmaf(a.x, b.x, fmaf(a.y, b.y, x));
    }
    return ex2(__fsub_rn(__fmul_rn(x, sc), offset));
}

template <int D, int DT, int NWG>
__global__ void __launch_bounds__(Cfg<D, NWG>::THREADS, Cfg<D, NWG>::PER_SM)
    k_attention_tc(const __grid_constant__ AttnArgs a) {
    using C = Cfg<D, NWG>;
    constexpr int ROWS = C::ROWS, H = C::H, SLOTS = C::SLOTS;
    extern __shared__ unsigned char raw[];
    unsigned char *sq = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    unsigned char *ring = sq + NWG * C::QTILE;
    Line &ln = *reinterpret_cast<Line *>(ring + SLOTS * C::TILE);
    Ctl &ctl = *reinterpret_cast<Ctl *>(&ln + 1);
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const prox_cache &c = a.cache;
    const int ps = c.page_size, sh = 31 - __clz(ps), G = a.n_heads / c.n_kv_heads;

    if (tid == 0) {
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(&ctl.full[i], 1);
            mbar_init(&ctl.empty[i], NWG);
        }
        for (int w = 0; w < NWG; ++w) {
            mbar_init(&ctl.q_ready[w], 4);
            mbar_init(&ctl.o_done[w], 1);
            mbar_init(&ctl.o_full[w], 1);
            mbar_init(&ctl.drained[w], 1);
            for (int b = 0; b < 2; ++b) {
                mbar_init(&ctl.s_full[w][b], 1);
                mbar_init(&ctl.p_ready[w][b], 4);
            }
        }
        ctl.dead = 0;
        for (int i = 0; i < 8; ++i) ctl.poison[i >> 2][i & 3] = 0;
        mbar_fence_init();
    }
    if (wid == 4 * NWG) tmem_alloc(&ctl.tmem, C::COLS);
    if (wid == 5 * NWG && lane < 2)
        asm volatile("prefetch.tensormap [%0];" ::"l"(
                         reinterpret_cast<uint64_t>(lane ? &a.map_v : &a.map_k))
                     : "memory");
    pdl_wait();
    pdl_launch();
    prefetch_queries(a, D);
    tc_fence_before();
    build_line(ln, a, ROWS, blockIdx.x == 0);  // (its barriers cover the setup above)
    tc_fence_after();
    const uint32_t tmem = ctl.tmem;
    const uint32_t t_s = tmem, t_o = tmem + NWG * 128;  // + 128 per row group
    const int run = run_length(ln, a.n, a.grid), total = ln.pre[a.n];
    const bool idle = total == 0 || blockIdx.x > (total - 1) / run;
    const int begin = idle ? 0 : blockIdx.x * run, end = idle ? 0 : begin + min(run, total - begin);
    const int per_box = min(ps, kKT), boxes = kKT / per_box;
    bool live = true;

    if (wid == 5 * NWG) {
        // ------------------------------------------------------------------
        // loading warp: lane = (page of the tile, 64 elements); the order of
        // slots is that of use: k0, k1, v0, k2, v1, ..., v last
        // ------------------------------------------------------------------
        const uint64_t policy = l2_evict_first();
        const int pg = lane / H, half = lane % H;
        int it = 0;
        for (int pos = begin; pos < end && live;) {
            const Stretch st = stretch_at(ln, a, ROWS, pos, end);
            pos += st.n_tiles;
            const int tot = ln.tot[st.b];
            const int32_t *table = c.page_table + (size_t)max(ln.seq[st.b], 0) * c.max_pages;
            auto page_of = [&](int tile) {
                const int key = tile * kKT + pg * per_box;
                return pg < boxes && key < tot ? table[key >> sh] : kNone;
            };
            // one tile of k or v into the next slot
            auto load = [&](const CUtensorMap *map, int tile, int page) {
                const int slot = it % SLOTS;
                if (!__all_sync(0xffffffffu, it < SLOTS || mbar_spin(&ctl.empty[slot], (it / SLOTS - 1) & 1,
                                                                     a.wait_us, &ctl.dead))) {
                    live = false;
                    ctl.dead = 1;
                    if (lane == 0) atomicOr(c.status, PROX_CACHE_TIMEOUT);
                    return;
                }
                // a page id out of range: zeros (a box outside the map), and the mask
                const bool wanted = page != kNone, good = page_ok(c, page);
                const unsigned load = __ballot_sync(0xffffffffu, wanted);
                const int y = good ? (page * c.n_kv_heads + st.head) * ps + (tile * kKT & (ps - 1))
                                   : c.n_pages * c.n_kv_heads * ps;
                if (wanted && !good) atomicOr(c.status, PROX_CACHE_BAD_STATE);
                const bool skip = blockIdx.x == 0 && it == a.debug_skip;
                if (lane == 0 && !skip)
                    mbar_arrive_expect_tx(&ctl.full[slot], __popc(load) * per_box * 128);
                __syncwarp();
                if (wanted && !skip)
                    box_g2s(smem_addr(ring) + slot * C::TILE + half * C::HALF + pg * per_box * 128,
                            map, half * 64, y, &ctl.full[slot], policy);
                ++it;
            };
            int now = page_of(st.tile0), next = kNone;
            load(&a.map_k, st.tile0, now);
            for (int i = 0; i < st.n_tiles && live; ++i) {
                const int tile = st.tile0 + i;
                if (i + 1 < st.n_tiles) {
                    next = page_of(tile + 1);
                    load(&a.map_k, tile + 1, next);
                }
                if (live) load(&a.map_v, tile, now);
                now = next;
            }
        }
        // no copy is in flight when the CTA ends, not behind a wait that gave up either
        // (whatever its bound was)
        for (int k = max(0, it - SLOTS); k < it; ++k)
            if (blockIdx.x > 0 || k != a.debug_skip)
                mbar_spin(&ctl.full[k % SLOTS], (k / SLOTS) & 1, kDefaultWaitUs);
    } else if (wid >= 4 * NWG) {
        // ------------------------------------------------------------------
        // a warp that issues a row group's MMAs: one elected thread does, but the
        // whole warp runs the loops on values it knows to be uniform, so that
        // operand descriptors live in uniform registers (computed by one thread
        // alone, an MMA took 90 cycles to issue); after a wait that gave up nothing
        // more is issued
        // ------------------------------------------------------------------
        const int w = NWG == 2 ? uniform(wid - 4 * NWG) : 0;
        constexpr uint32_t qk_idesc = idesc_of<DT>(kKT, false), pv_idesc = idesc_of<DT>(D, true);
        // low words of the descriptors of the first q, k and v tiles (the address
        // field, in 16 bytes, never carries); the high words are constants
        const uint32_t q_lo = uniform((uint32_t)sw128_desc(smem_addr(sq), 16, 1024)),
                       k_lo = uniform((uint32_t)sw128_desc(smem_addr(ring), 16, 1024)),
                       v_lo = uniform((uint32_t)sw128_desc(smem_addr(ring), C::HALF, 1024));
        constexpr uint64_t hi = (uint64_t)(1024u >> 4) << 32 | 1ull << 46 | 2ull << 61;
        const uint32_t d_s = uniform(t_s + w * 128), d_o = uniform(t_o + w * 128);
        const uint32_t q0 = q_lo + w * (C::QTILE >> 4);
        const bool one = elect_one();
        uint32_t n_q = 0, n_s = 0, n_p = 0;  // stretches, scores formed, probabilities used
        int slot = 0, turn = 0;              // of the next slot in the order of loading
        auto await = [&] { wait_or_give_up(&ctl.full[slot], turn, a, ctl, live); };
        auto next = [&] {
            if (++slot == SLOTS) {
                slot = 0;
                ++turn;
            }
        };
        // scores of the slot's tile (there already), into the next buffer
        auto qk = [&] {
            const uint32_t d = d_s + (n_s & 1) * 64;
            const uint32_t k0 = k_lo + slot * (C::TILE >> 4);
            if (one && live) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    umma(d, hi | (q0 + (k / 4) * (C::QHALF >> 4) + (k % 4) * 2),
                         hi | (k0 + (k / 4) * (C::HALF >> 4) + (k % 4) * 2), qk_idesc, k > 0);
                umma_commit(&ctl.s_full[w][n_s & 1]);
                umma_commit(&ctl.empty[slot]);
            }
            ++n_s;
            next();
        };
        for (int pos = begin; pos < end;) {
            const Stretch st = stretch_at(ln, a, ROWS, pos, end);
            pos += st.n_tiles;
            const int n_tiles = uniform(st.n_tiles);
            if (w == 1 && uniform(ln.rows[st.b] * G - st.row_tile * ROWS) <= 128) {
                // no rows of this group: the slots are the other one's alone
                for (int i = 0; i < 2 * n_tiles; ++i) {
                    await();
                    if (one && live) mbar_arrive(&ctl.empty[slot]);
                    next();
                }
                continue;
            }
            // scores of tiles 0 and 1, then the product with v of tile i and, into
            // the score buffer that it frees, the scores of tile i + 2
            wait_or_give_up(&ctl.q_ready[w], n_q++, a, ctl, live);
            for (int i = 0; i < min(n_tiles, 2); ++i) {
                await();
                tc_fence_after();
                qk();
            }
            for (int i = 0; i < n_tiles; ++i) {
                const uint32_t buf = n_p & 1, v0 = v_lo + slot * (C::TILE >> 4);
                const bool more = i + 2 < n_tiles;
                // (a wait takes 120 cycles even when it is over: those for memory
                // come first, so that only one lies behind the softmax)
                uint64_t *v_free = &ctl.empty[slot];
                await();
                next();
                if (more) await();
                wait_or_give_up(&ctl.p_ready[w][buf], n_p >> 1, a, ctl, live);
                ++n_p;
                tc_fence_after();
                if (one && live) {
#pragma unroll
                    for (int k = 0; k < kKT / 16; ++k)
                        umma_ts(d_o, d_s + buf * 64 + k * 8, hi | (v0 + k * (2048 >> 4)), pv_idesc,
                                k > 0 || i > 0);
                    if (i + 2 == n_tiles || n_tiles == 1) umma_commit(&ctl.o_done[w]);
                    if (i + 1 == n_tiles) umma_commit(&ctl.o_full[w]);
                }
                if (more) qk();
                if (one && live) umma_commit(v_free);
            }
        }
        // The MMAs issued come to their end before the tensor memory is freed. (The
        // softmax has waited for them already, unless a wait of its own gave up.)
        if (one && n_s > 0) {
            umma_commit(&ctl.drained[w]);
            mbar_spin(&ctl.drained[w], 0, kDefaultWaitUs);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------------
        // softmax: row group w, one thread a row
        // ------------------------------------------------------------------
        const int w = wid >> 2, t = tid & 127;
        const uint32_t lane_at = (uint32_t)(wid & 3) << 21;   // first tensor-memory lane << 16
        const uint32_t to = t_o + w * 128 + lane_at;
        // tiles and stretches of the row group so far, slots used by all stretches
        uint32_t n = 0, n_full = 0, odd_stretch = 0;
        int it = 0;
        Stretch st = {};
        if (begin < end) st = stretch_at(ln, a, ROWS, begin, end);
        // A row of a stretch's tile: its drafted token and head, whether it exists. Worked
        // out anew where it is wanted (q, masks, outputs): kept over the loop of tiles, it
        // took registers that the scores then had to leave for local memory (16 sequences
        // of 8,000 to 32,000 tokens in short runs: 427 -> 401 us at the time). With one row
        // group there is room for the token alone, which spares short units a division
        // (ragged batch 41.9 -> 40.3).
        struct Place {
            int tok, head;
            size_t row;
            const uint64_t *tree;
            bool there;
        };
        auto token = [&](const Stretch &s, int rt) {
            const int r = s.row_tile * ROWS + rt;
            return r < ln.rows[s.b] * G ? r / G : 0;
        };
        auto place = [&](const Stretch &s, int rt, int tok) {
            Place p;
            const int r = s.row_tile * ROWS + rt;
            p.there = r < ln.rows[s.b] * G;
            p.tok = tok;
            p.head = s.head * G + (p.there ? r - p.tok * G : 0);
            p.row = (size_t)ln.row0[s.b] + p.tok;
            p.tree = a.tree ? a.tree + p.row * a.tree_words : nullptr;
            return p;
        };
        for (int pos = begin; pos < end;) {
            const bool first = pos == begin;
            pos += st.n_tiles;
            const int n_rows = ln.rows[st.b] * G - st.row_tile * ROWS;  // of this row tile
            named_bar_sync(2, C::SOFT);  // all are done with the notes of the last stretch
            if (w * 128 >= n_rows) {
                odd_stretch ^= 1;
                it += 2 * st.n_tiles;
                if (pos < end) st = stretch_at(ln, a, ROWS, pos, end);
                continue;
            }
            // this stretch's notes; the next one's are cleared
            odd_stretch ^= 1;
            if (tid < 4) ctl.poison[odd_stretch][tid] = 0;
            auto poison = [&]() -> uint64_t * { return ctl.poison[odd_stretch ^ 1]; };
            const int rt = w * 128 + t;                  // row of the tile
            const int tok = token(st, rt);
            const bool busy = rt - lane < n_rows;        // the warp has rows
            {
                const Place me = place(st, rt, tok);
                // q: the warp's 32 rows, a row's 16-byte pieces side by side (each lane
                // knows where its own row is); rows behind the last one are zeros
                constexpr int P = D / 8, PER = 32 / P;  // pieces of a row, rows a step
                const int64_t mine_at =
                    me.there ? (int64_t)me.row * a.q_stride + (int64_t)me.head * D : -1;
                unsigned char *dst = sq + w * C::QTILE + (t - lane) * 128;
                if (busy) {
                    uint4 v[P];
#pragma unroll
                    for (int y = 0; y < P; ++y) {
                        const int64_t from = __shfl_sync(0xffffffffu, mine_at, y * PER + lane / P);
                        v[y] = from >= 0 ? reinterpret_cast<const uint4 *>(a.q + from)[lane % P]
                                         : make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int y = 0; y < P; ++y) {
                        const int k = y * PER + lane / P, x = lane % P;
                        *reinterpret_cast<uint4 *>(dst + k * 128 + (x >> 3) * C::QHALF +
                                                   (((x & 7) ^ (k & 7)) << 4)) = v[y];
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.q_ready[w]);
            }
            // pages with an id out of range, a bit each, of the next 32 / boxes tiles
            const int span = 32 / boxes;
            int first_edge = ln.len[st.b] / kKT - st.tile0;  // first tile with drafted or missing keys
            uint32_t unreadable = 0;
            int looked = 0;
            auto look = [&](int i) {
                const int key = (st.tile0 + i) * kKT + lane * per_box;
                const bool in = i + lane / boxes < st.n_tiles && key < ln.tot[st.b];
                const int32_t *table = c.page_table + (size_t)max(ln.seq[st.b], 0) * c.max_pages;
                unreadable = __ballot_sync(0xffffffffu, in && !page_ok(c, table[key >> sh]));
                looked = i;
            };
            look(0);
            float m = -INFINITY, l = 0.f;         // offset in use (log2 units) and sum
            uint32_t s0[32], s1[32];              // scores
            // what the scores are multiplied with on their way into e^x: 1 once a row of
            // the warp has an offset beyond kRoundFirst, they are scaled themselves then
            float by = a.scale_log2;
            // tile i's buffer; its scores are there after the wait
            auto buffer = [&](int i) { return t_s + w * 128 + ((n + i) & 1) * 64 + lane_at; };
            auto formed = [&](int i) {
                wait_or_give_up(&ctl.s_full[w][(n + i) & 1], (n + i) >> 1, a, ctl, live);
                tc_fence_after();
            };
            formed(0);
            if (busy) tmem_ask32(buffer(0), s0);
            for (int i = 0; i < st.n_tiles; ++i) {
                const int tile = st.tile0 + i;
                const uint32_t ts = buffer(i);
                if (busy) {
                    tmem_ask32(ts + 32, s1);
                    tmem_take32(s0);
                    tmem_take32(s1);
                }
                if (i - looked >= span) look(i);
                const uint32_t bad = unreadable >> ((i - looked) * boxes) & ((1u << boxes) - 1);
                const bool edge = i >= first_edge;       // (tile + 1) * kKT > committed tokens
                if (edge) {
                    const int len = ln.len[st.b], tot = ln.tot[st.b];
                    // v's rows that must not meet the tensor core, two threads a
                    // key: rows behind the last key (0 * inf is not 0), and the
                    // infinities and NaN of drafted tokens, which only some rows
                    // see; those come back when the outputs are written. (Each row
                    // group does it before its own product, to the same effect; what
                    // was found is noted before it is taken out.)
                    const int kr = t & (kKT - 1), key = tile * kKT + kr;
                    const int at = it + (i + 1 < st.n_tiles ? 2 * i + 2 : 2 * i + 1), slot = at % SLOTS;
                    wait_or_give_up(&ctl.full[slot], at / SLOTS, a, ctl, live);
                    // (pieces in an order that keeps a warp's rows on different banks)
                    constexpr int P = D / 16;
                    unsigned char *vr = ring + slot * C::TILE + kr * 128;
                    auto piece_at = [&](int x) {
                        const int y = (t >> 6) * P + x;
                        return reinterpret_cast<uint4 *>(vr + (y >> 3) * C::HALF +
                                                         (((y & 7) ^ (kr & 7)) << 4));
                    };
                    if (key >= tot) {
#pragma unroll
                        for (int x = 0; x < P; ++x) *piece_at(x) = make_uint4(0, 0, 0, 0);
                    } else if (key >= len) {
                        uint4 v[P];
                        bool odd = false;
#pragma unroll
                        for (int x = 0; x < P; ++x) v[x] = *piece_at(x);
#pragma unroll
                        for (int x = 0; x < P; ++x)
                            odd |= non_finite2<DT>(v[x].x) || non_finite2<DT>(v[x].y) ||
                                   non_finite2<DT>(v[x].z) || non_finite2<DT>(v[x].w);
                        if (odd) {
                            atomicOr(reinterpret_cast<unsigned long long *>(
                                         &poison()[(key - len) >> 6 & 3]),
                                     1ull << (key - len & 63));
                            __threadfence_block();
#pragma unroll 1
                            for (int x = 0; x < P; ++x) {
                                const uint4 u = *piece_at(x);
                                *piece_at(x) = make_uint4(finite2<DT>(u.x), finite2<DT>(u.y),
                                                          finite2<DT>(u.z), finite2<DT>(u.w));
                            }
                        }
                    }
                    fence_proxy_async_smem();
                }
                if (busy) {
                    // scores not seen are -inf
                    auto mask = [&](uint32_t bits, uint32_t(&s)[32]) {
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            if (!(bits >> x & 1)) s[x] = 0xff800000u;
                    };
                    // (once, but for the tile in which a row's offset passes kRoundFirst)
                    for (;;) {
                        if (i >= first_edge || bad) {
                            const Place me = place(st, rt, NWG == 1 ? tok : token(st, rt));
                            uint64_t seen = low_bits(ln.tot[st.b] - tile * kKT);
                            for (int p = 0; p < boxes; ++p)
                                if (bad >> p & 1) seen &= ~(low_bits(per_box) << (p * per_box));
                            seen = me.there ? seen_bits(me.tree, a.tree_words, ln.len[st.b], me.tok, tile * kKT) & seen
                                            : 0ull;
                            mask((uint32_t)seen, s0);
                            mask((uint32_t)(seen >> 32), s1);
                            if (by != a.scale_log2) {
#pragma unroll
                                for (int x = 0; x < 32; ++x) {
                                    s0[x] = __float_as_uint(__fmul_rn(__uint_as_float(s0[x]), a.scale_log2));
                                    s1[x] = __float_as_uint(__fmul_rn(__uint_as_float(s1[x]), a.scale_log2));
                                }
                            }
                        }
                        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            mx[x & 3] = fmaxf(mx[x & 3], fmaxf(__uint_as_float(s0[x]), __uint_as_float(s1[x])));
                        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * by;
                        if (!__any_sync(0xffffffffu, top > m + kGrow || (top > m && m == -INFINITY))) break;
                        const float nm = fmaxf(m, top);
                        if (by != 1.f && __any_sync(0xffffffffu, fabsf(nm) >= kRoundFirst && nm != -INFINITY)) {
                            by = 1.f;
                            first_edge = min(first_edge, i);  // (and on to the branch above from here on)
                            continue;
                        }
                        const float f = nm > m ? ex2(m - nm) : 1.f;
                        m = nm;
                        l *= f;
                        if (i > 0) {
                            // The last tile's product is in the outputs once the next
                            // tile's scores are formed, which come behind it.
                            if (i + 1 < st.n_tiles) {
                                formed(i + 1);
                            } else {
                                wait_or_give_up(&ctl.o_done[w], n_full, a, ctl, live);
                                tc_fence_after();
                            }
#pragma unroll 1
                            for (int q = 0; q < D / 16; ++q) {
                                uint32_t o[16];
                                tmem_ld16(to + q * 16, o);
#pragma unroll
                                for (int x = 0; x < 16; ++x)
                                    o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
                                tmem_st16(to + q * 16, o);
                            }
                        }
                        break;
                    }
                    const float mu = m == -INFINITY ? 0.f : m;
                    const float2 sc2 = make_float2(by, by), mu2 = make_float2(-mu, -mu);
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    auto probabilities = [&](const uint32_t(&s)[32], uint32_t at) {
                        uint32_t p[16];
#pragma unroll
                        for (int x = 0; x < 32; x += 2) {
                            const float2 z = fma2(
                                make_float2(__uint_as_float(s[x]), __uint_as_float(s[x + 1])), sc2, mu2);
                            const float2 e = make_float2(ex2(z.x), ex2(z.y));
                            sum[x / 2 & 1] = add2(sum[x / 2 & 1], e);
                            p[x / 2] = pack2<DT>(e.x, e.y);
                        }
                        tmem_st16(at, p);
                    };
                    probabilities(s0, ts);
                    if (i + 1 < st.n_tiles) {
                        formed(i + 1);
                        tmem_ask32(buffer(i + 1), s0);
                    }
                    probabilities(s1, ts + 16);
                    sum[0] = add2(sum[0], sum[1]);
                    l += sum[0].x + sum[0].y;
                    tmem_st_wait();
                }
                else if (i + 1 < st.n_tiles) {
                    formed(i + 1);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.p_ready[w][(n + i) & 1]);
            }
            it += 2 * st.n_tiles;
            n += st.n_tiles;
            // --------------------------------------------------------------
            // the rows' outputs, or a piece of them
            // --------------------------------------------------------------
            const Stretch now = st;
            if (pos < end) st = stretch_at(ln, a, ROWS, pos, end);  // (while there is time)
            if (blockIdx.x == 0 && (int)n_full == a.debug_give_up) {
                live = false;
                ctl.dead = 1;
                atomicOr(c.status, PROX_CACHE_TIMEOUT);
            }
            // (a wait tells a phase by its parity, so every phase is waited for)
            wait_or_give_up(&ctl.o_done[w], n_full, a, ctl, live);
            wait_or_give_up(&ctl.o_full[w], n_full++, a, ctl, live);
            tc_fence_after();
            if (busy) {
                const bool whole = now.n_tiles == now.all_tiles;
                const float inv = l == 0.f ? 0.f : whole ? 1.f / l : 1.f;
                float *part = piece(a, blockIdx.x, first, D, ROWS);
                const Place me = place(now, rt, NWG == 1 ? tok : token(now, rt));
                const uint64_t *odd = poison(), any = odd[0] | odd[1] | odd[2] | odd[3];
#pragma unroll 1
                for (int q = 0; q < D / 32; ++q) {
                    uint32_t ob[32];
                    tmem_get32(to + q * 32, ob);
                    float o[32];
#pragma unroll
                    for (int x = 0; x < 32; ++x) o[x] = __uint_as_float(ob[x]) * inv;
                    if (any && me.there) {
                        for (int k = 0; k < 4; ++k) {
                            uint64_t bits = odd[k];
                            bits &= me.tree ? (k < a.tree_words ? me.tree[k] : 0ull)
                                            : low_bits(me.tok + 1 - k * 64);
                            for (; bits; bits &= bits - 1) {
                                const int key = ln.len[now.b] + k * 64 + __ffsll((long long)bits) - 1;
                                const int page =
                                    c.page_table[(size_t)ln.seq[now.b] * c.max_pages + (key >> sh)];
                                if (!page_ok(c, page)) continue;  // (cannot be: its box was read)
                                const size_t at =
                                    (((size_t)page * c.n_kv_heads + now.head) * ps + (key & (ps - 1))) * D;
                                // p v, so that an infinity without weight is NaN here as in
                                // k_attention.cu (the finite elements of the row are in o)
                                const float p = draft_weight<D, DT>(
                                    sq + w * C::QTILE, t, c.k + (a.v_layer - c.v) + at, a.scale_log2, m);
                                const uint32_t *v =
                                    reinterpret_cast<const uint32_t *>(a.v_layer + at + q * 32);
#pragma unroll
                                for (int x = 0; x < 32; x += 2) {
                                    const uint32_t vv = v[x / 2];
                                    if (!non_finite2<DT>(vv)) continue;
                                    const float2 f = unpack2<DT>(vv);
                                    if (!isfinite(f.x)) o[x] += p * f.x;
                                    if (!isfinite(f.y)) o[x + 1] += p * f.y;
                                }
                            }
                        }
                    }
                    if (any) __syncwarp();  // (the next columns' load wants the warp together)
                    if (!whole) {
#pragma unroll
                        for (int x = 0; x < 32; x += 4)
                            reinterpret_cast<float4 *>(part)[(size_t)(q * 8 + x / 4) * ROWS + rt] =
                                make_float4(o[x], o[x + 1], o[x + 2], o[x + 3]);
                    } else if (me.there) {
                        uint4 *op = reinterpret_cast<uint4 *>(a.out + me.row * a.out_stride +
                                                              (size_t)me.head * D + q * 32);
#pragma unroll
                        for (int x = 0; x < 32; x += 8)
                            op[x / 8] = make_uint4(pack2<DT>(o[x], o[x + 1]), pack2<DT>(o[x + 2], o[x + 3]),
                                                   pack2<DT>(o[x + 4], o[x + 5]),
                                                   pack2<DT>(o[x + 6], o[x + 7]));
                    }
                }
                if (!whole) {
                    part[ROWS * D + rt] = m;
                    part[ROWS * (D + 1) + rt] = l;
                } else if (me.there && a.lse) {
                    a.lse[me.row * a.n_heads + me.head] =
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
    static_assert(Cfg<D, NWG>::PER_SM * (smem + 1024) <= 228 * 1024, "shared memory of an SM");
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
