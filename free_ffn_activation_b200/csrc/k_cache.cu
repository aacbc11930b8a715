// Page operations of the paged key/value cache (include/prox_decode.h).
//
// Bookkeeping (reserve, fork, free) runs in one cluster of CTAs: the
// entries' page counts are prefix-summed by every CTA for itself, so each
// entry's place on the free list is known without atomics and the result does
// not depend on timing, and the pages are then handled in chunks of 32 columns
// dealt out to the cluster's warps. Decisions are taken from lengths, page
// counts and the free count, which are written behind a cluster barrier only.
// These kernels are bound by latency: a chain of dependent reads and barriers.
// The rows themselves are moved by kernels over the whole GPU (fork's copies,
// append, compact), a warp or a group of lanes per run of rows.
#include "decode_internal.cuh"

#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <cstdint>
#include <mutex>

namespace cg = cooperative_groups;

namespace prox {
namespace {

// Shapes of a bookkeeping call: few entries that can list few pages (by the page
// table's width) run on 8 CTAs of 256 threads, others on 16 of 1024. Fork and
// free on the device (us; 8 of 256 | 16 of 1024), by entries x pages of each:
//   8 x 50      15.5 |  17.6     32 x 50     16.0 | 19.8     128 x 20    19.4 | 20.4
//   8 x 200     16.1 |  18.6     32 x 250    25.5 | 19.4     128 x 100   38.6 | 20.2
//   8 x 1,000   23.7 |  19.2     32 x 500    36.4 | 19.6     256 x 4     25.9 | 19.7
//   8 x 2,000   32.6 |  19.8     32 x 2,500 115.6 | 31.1     256 x 64    38.7 | 20.4
// The shapes cross between 2,600 and 8,000 pages, and by 256 entries for any pages.
// (A wide table of short sequences costs the larger shape's 2 us, a full one of 16,000
// pages cost the smaller one 16.)
constexpr int kFew = 256;              // entries that the smaller shape has room for
constexpr int kFewEntries = 128, kFewPages = 4096, kFewCtas = 8;
constexpr int kSome = 1024, kCtas = 16;
constexpr int kWindow = 8192;          // chunks of a CTA whose owners and masks are kept

// exclusive prefix sum over the block (and the total), v per thread
template <int THREADS, typename T>
__device__ T block_scan(T v, T *tmp, T *total) {
    constexpr int WARPS = THREADS / 32;
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    T x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) tmp[wid] = x;
    __syncthreads();
    // every warp sums the warps for itself
    T w = lane < WARPS ? tmp[lane] : T(0);
#pragma unroll
    for (int o = 1; o < WARPS; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    *total = __shfl_sync(0xffffffffu, w, WARPS - 1);
    const T base = __shfl_sync(0xffffffffu, w, wid ? wid - 1 : 0);
    return (wid ? base : T(0)) + x - v;
}

// shared memory of a bookkeeping CTA of N entries at most: `first` finds
// sequences listed twice, the others hold what each entry needs
template <int N>
struct Book {
    int seq[N];          // sequence of the entry, -1 = left out
    int aux[N];          // fork: source; reserve: columns held so far
    int len[N];          // fork: the source's length
    int cols[N];         // columns (pages) the entry works on
    int base[N];         // pages taken by the entries before it
    int chunk[N + 1];    // chunks of 32 columns before it
    int tmp[32];
    long long wide[32];
    int count;           // free: pages given back by this CTA
    int odd;             // free: a count was 0 already
    int first[kMaxSeqs]; // lowest entry that lists the sequence (max_seqs of them)
};

// entry whose chunks contain chunk c: the last i with chunk[i] <= c
__device__ __forceinline__ int find_entry(const int *chunk, int n, int c) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (chunk[mid] <= c)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// marks each sequence's first listing (all threads; ends with a barrier)
template <int THREADS>
__device__ void find_first(const prox_cache &c, int *first, const int32_t *seqs, int n) {
    for (int s = threadIdx.x; s < c.max_seqs; s += THREADS) first[s] = 0x7fffffff;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += THREADS) {
        const int s = seqs[i];
        if (s >= 0 && s < c.max_seqs) atomicMin(&first[s], i);
    }
    __syncthreads();
}

// exclusive sums of chunks of 32 columns over the entries; returns their count
// (ends with a barrier)
template <int THREADS, int N>
__device__ int sum_chunks(Book<N> &b, int n) {
    constexpr int PER = N / THREADS;
    const int i0 = threadIdx.x * PER;
    int mine = 0, total;
    for (int k = 0; k < PER; ++k)
        if (i0 + k < n) mine += (b.cols[i0 + k] + 31) >> 5;
    int at = block_scan<THREADS>(mine, b.tmp, &total);
    for (int k = 0; k < PER; ++k)
        if (i0 + k < n) {
            b.chunk[i0 + k] = at;
            at += (b.cols[i0 + k] + 31) >> 5;
        }
    __syncthreads();
    return total;
}

// Which entries get their pages: an entry that needs none always does, the
// others as long as the sum up to and with them fits in the free list. need
// comes from `need_of(i)` (-1: refused for another reason). base[] gets the
// pages taken before the entry; returns the pages taken in all.
template <int THREADS, int N, typename F>
__device__ int take_pages(Book<N> &b, int n, int n_free, uint32_t *status, bool *fits, F need_of) {
    // (sums in 64 bits: refused entries may ask for more pages than there are)
    constexpr int PER = N / THREADS;
    const int i0 = threadIdx.x * PER;
    int need[PER];
    long long mine = 0, total;
    for (int k = 0; k < PER; ++k) {
        need[k] = i0 + k < n ? need_of(i0 + k) : -1;
        mine += max(need[k], 0);
    }
    long long at = block_scan<THREADS>(mine, b.wide, &total);
    if (threadIdx.x == 0) b.count = 0;
    __syncthreads();
    int taken = 0;
    for (int k = 0; k < PER; ++k) {
        if (i0 + k >= n) continue;
        const bool ok = need[k] == 0 || (need[k] > 0 && at + need[k] <= n_free);
        b.base[i0 + k] = ok ? (int)min(at, (long long)n_free) : 0;
        fits[k] = ok;
        if (need[k] > 0) {
            at += need[k];
            if (ok)
                taken = (int)at;
            else
                atomicOr(status, PROX_CACHE_FULL);
        }
    }
    // entries that fit and need pages come first: the largest end is the sum
    taken = __reduce_max_sync(0xffffffffu, taken);
    if ((threadIdx.x & 31) == 0 && taken > 0) atomicMax(&b.count, taken);
    __syncthreads();
    return b.count;
}

__device__ __forceinline__ int free_count(const prox_cache &c) {
    const int f = *c.n_free;
    if (f < 0 || f > c.n_pages) atomicOr(c.status, PROX_CACHE_BAD_STATE);
    return min(max(f, 0), c.n_pages);
}

// the k-th page taken from a free list of n_free pages; -1 (and the status
// bit) where the list holds no page id or one that is in use
__device__ __forceinline__ int pop_page(const prox_cache &c, int n_free, int k) {
    const int p = c.free_list[n_free - 1 - k];
    if (page_ok(c, p) && c.ref_count[p] == 0) {
        c.ref_count[p] = 1;
        return p;
    }
    atomicOr(c.status, PROX_CACHE_BAD_STATE);
    return -1;
}

__global__ void __launch_bounds__(256) k_cache_init(const prox_cache c) {
    pdl_wait();
    pdl_launch();
    const int stride = gridDim.x * blockDim.x, t = blockIdx.x * blockDim.x + threadIdx.x;
    for (int p = t; p < c.n_pages; p += stride) {
        c.ref_count[p] = 0;
        c.free_list[p] = c.n_pages - 1 - p;
    }
    for (int s = t; s < c.max_seqs; s += stride) c.length[s] = c.held[s] = 0;
    if (t == 0) {
        *c.n_free = c.n_pages;
        *c.status = 0;
    }
}

__global__ void k_cache_clear(const prox_cache c, uint32_t bits) {
    pdl_wait();
    pdl_launch();
    atomicAnd(c.status, ~bits);
}

// ---------------------------------------------------------------------------
// reserve
// ---------------------------------------------------------------------------
template <int THREADS, int N>
__global__ void __launch_bounds__(THREADS)
    k_cache_reserve(const prox_cache c, int n, const int32_t *seqs, const int32_t *n_new,
                    uint8_t *ok_out) {
    extern __shared__ __align__(16) unsigned char smem[];
    Book<N> &b = *reinterpret_cast<Book<N> *>(smem);
    cg::cluster_group cl = cg::this_cluster();
    const int rank = cl.block_rank();
    pdl_wait();
    pdl_launch();
    const int n_free = free_count(c);
    find_first<THREADS>(c, b.first, seqs, n);
    bool fits[N / THREADS];
    const int taken = take_pages<THREADS>(b, n, n_free, c.status, fits, [&](int i) {
        const int s = entry_seq(c, seqs, i);
        b.seq[i] = -1;
        b.cols[i] = 0;
        if (s < 0) return -1;
        if (b.first[s] != i) {
            atomicOr(c.status, PROX_CACHE_BAD_SEQ);
            return -1;
        }
        const int add = n_new[i];
        if (add < 0) {
            atomicOr(c.status, PROX_CACHE_BAD_ARG);
            return -1;
        }
        const SeqState st = seq_state(c, s);
        const long want = ((long)st.len + add + c.page_size - 1) / c.page_size;
        if (want > c.max_pages) {
            atomicOr(c.status, PROX_CACHE_FULL);
            return -1;
        }
        b.seq[i] = s;
        b.aux[i] = st.held;
        b.cols[i] = max(0, (int)want - st.held);
        return b.cols[i];
    });
    for (int k = 0; k < N / THREADS; ++k) {
        const int i = threadIdx.x * (N / THREADS) + k;
        if (i >= n) continue;
        if (!fits[k]) {
            b.seq[i] = -1;
            b.cols[i] = 0;
        }
        if (rank == 0 && ok_out) ok_out[i] = fits[k] ? 1 : 0;
    }
    const int chunks = sum_chunks<THREADS>(b, n);
    const int lane = threadIdx.x & 31;
    for (int q = rank * (THREADS / 32) + (threadIdx.x >> 5); q < chunks; q += cl.num_blocks() * (THREADS / 32)) {
        const int i = find_entry(b.chunk, n, q);
        const int j = (q - b.chunk[i]) * 32 + lane;
        if (j >= b.cols[i]) continue;
        c.page_table[(size_t)b.seq[i] * c.max_pages + b.aux[i] + j] =
            pop_page(c, n_free, b.base[i] + j);
    }
    cl.sync();  // every CTA has read the state
    if (rank == 0) {
        for (int i = threadIdx.x; i < n; i += THREADS)
            if (b.seq[i] >= 0 && b.cols[i] > 0) c.held[b.seq[i]] = b.aux[i] + b.cols[i];
        if (threadIdx.x == 0) *c.n_free = n_free - taken;
    }
}

// ---------------------------------------------------------------------------
// fork
// ---------------------------------------------------------------------------
// ws: [0] = page copies, then {source page, target page, rows, -} for each
template <int THREADS, int N>
__global__ void __launch_bounds__(THREADS)
    k_cache_fork(const prox_cache c, int n, const int32_t *src, const int32_t *dst, int share,
                 uint8_t *ok_out, int32_t *ws) {
    extern __shared__ __align__(16) unsigned char smem[];
    Book<N> &b = *reinterpret_cast<Book<N> *>(smem);
    cg::cluster_group cl = cg::this_cluster();
    const int rank = cl.block_rank(), ps = c.page_size;
    pdl_wait();
    pdl_launch();
    const int n_free = free_count(c);
    find_first<THREADS>(c, b.first, dst, n);
    bool fits[N / THREADS];
    const int taken = take_pages<THREADS>(b, n, n_free, c.status, fits, [&](int i) {
        const int d = entry_seq(c, dst, i), s = entry_seq(c, src, i);
        b.seq[i] = -1;
        b.cols[i] = 0;
        if (d < 0) return -1;
        if (b.first[d] != i) {
            atomicOr(c.status, PROX_CACHE_BAD_SEQ);
            return -1;
        }
        if (s < 0) return -1;
        const int dl = c.length[d], dh = c.held[d], l = seq_state(c, s).len;
        if (dl != 0 || dh != 0) {
            atomicOr(c.status, PROX_CACHE_BAD_ARG);
            return -1;
        }
        b.seq[i] = d;
        b.aux[i] = s;
        b.len[i] = l;
        b.cols[i] = (l + ps - 1) / ps;
        return share ? (l % ps ? 1 : 0) : b.cols[i];
    });
    for (int k = 0; k < N / THREADS; ++k) {
        const int i = threadIdx.x * (N / THREADS) + k;
        if (i >= n) continue;
        if (!fits[k]) {
            b.seq[i] = -1;
            b.cols[i] = 0;
        }
        if (rank == 0 && ok_out) ok_out[i] = fits[k] ? 1 : 0;
    }
    const int chunks = sum_chunks<THREADS>(b, n);
    const int lane = threadIdx.x & 31;
    // two chunks a step, their reads in flight together
    constexpr int U = 2;
    const int step = (int)cl.num_blocks() * (THREADS / 32);
    for (int q0 = rank * (THREADS / 32) + (threadIdx.x >> 5); q0 < chunks; q0 += step * U) {
        int at[U], col[U], page[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int q = q0 + u * step;
            at[u] = q < chunks ? find_entry(b.chunk, n, q) : -1;
            if (at[u] >= 0) {
                col[u] = (q - b.chunk[at[u]]) * 32 + lane;
                if (col[u] >= b.cols[at[u]]) at[u] = -1;
            }
            if (at[u] >= 0)
                page[u] = c.page_table[(size_t)b.aux[at[u]] * c.max_pages + col[u]];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = at[u], j = col[u];
            if (i < 0) continue;
            const int rows = min(ps, b.len[i] - j * ps);
            int p = page[u];
            const bool good = page_ok(c, p);
            if (!good) atomicOr(c.status, PROX_CACHE_BAD_STATE);
            if (share && rows == ps) {
                if (good) atomicAdd(&c.ref_count[p], 1);
            } else {
                const int k = b.base[i] + (share ? 0 : j);
                const int to = pop_page(c, n_free, k);
                const int4 copy = make_int4(p, to, good && to >= 0 ? rows : 0, 0);
                reinterpret_cast<int4 *>(ws + 4)[k] = copy;
                p = to;
            }
            c.page_table[(size_t)b.seq[i] * c.max_pages + j] = p;
        }
    }
    cl.sync();  // every CTA has read the state
    if (rank == 0) {
        for (int i = threadIdx.x; i < n; i += THREADS)
            if (b.seq[i] >= 0) {
                c.length[b.seq[i]] = b.len[i];
                c.held[b.seq[i]] = b.cols[i];
            }
        if (threadIdx.x == 0) {
            *c.n_free = n_free - taken;
            ws[0] = taken;
        }
    }
}

// rows of the pages of fork's list, all layers: one warp moves the rows of one
// head of one page (contiguous), eight 16-byte pieces a lane in flight. Bound by
// memory: 3.7 GB read and written in 637 us together with its fork and free, 5.9 TB/s,
// 90% of the rate of a copy.
__global__ void __launch_bounds__(256) k_cache_copy(const prox_cache c, const int32_t *ws) {
    pdl_wait();
    pdl_launch();
    const int copies = ws[0];
    const int4 *list = reinterpret_cast<const int4 *>(ws + 4);
    const int lane = threadIdx.x & 31;
    const int per_row = c.head_dim / 8;                       // 16-byte pieces
    const long items = (long)copies * c.n_layers * 2 * c.n_kv_heads;
    const long step = (long)gridDim.x * (blockDim.x / 32);
    for (long it = (long)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5); it < items;
         it += step) {
        const int h = (int)(it % c.n_kv_heads);
        const long r = it / c.n_kv_heads;
        uint16_t *pool = r & 1 ? c.v : c.k;
        const long r2 = r >> 1;
        const int layer = (int)(r2 % c.n_layers);
        const int4 cp = list[r2 / c.n_layers];
        if (cp.z <= 0) continue;
        const size_t one = (size_t)c.page_size * c.head_dim;
        const uint4 *from = reinterpret_cast<const uint4 *>(
            pool + (((size_t)layer * c.n_pages + cp.x) * c.n_kv_heads + h) * one);
        uint4 *to = reinterpret_cast<uint4 *>(
            pool + (((size_t)layer * c.n_pages + cp.y) * c.n_kv_heads + h) * one);
        const int pieces = cp.z * per_row;
        for (int p = lane; p < pieces; p += 256) {
            uint4 v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (p + u * 32 < pieces) v[u] = __ldcs(from + p + u * 32);
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (p + u * 32 < pieces) __stcs(to + p + u * 32, v[u]);
        }
    }
}

// ---------------------------------------------------------------------------
// free
// ---------------------------------------------------------------------------
// A page's count, taken down by every listing, reaches 0 when nobody holds it
// any more. Its place on the free list is that of its first listing: once all
// counts are down, every listing of a page at 0 offers its number, and the
// smallest stays in the count (as a negative code far from any count) until
// the page is pushed.
constexpr int kClaim = (int)0x80000000;      // + listing number < 2^30
constexpr int kClaimEnd = kClaim + (1 << 30);

// A CTA's chunks are a run, so that pages come out in listing order. Which entry
// a chunk belongs to and which of its lanes push their page is kept for a window
// of chunks (all of them, up to two million pages a call).
struct Window {
    uint16_t owner[kWindow];
    uint32_t mask[kWindow];
    int before[kWindow];
};

template <int THREADS, int N>
__global__ void __launch_bounds__(THREADS)
    k_cache_free(const prox_cache c, int n, const int32_t *seqs) {
    extern __shared__ __align__(16) unsigned char smem[];
    Book<N> &b = *reinterpret_cast<Book<N> *>(smem);
    Window &w = *reinterpret_cast<Window *>(smem + (sizeof(Book<N>) + 15) / 16 * 16);
    cg::cluster_group cl = cg::this_cluster();
    const int rank = cl.block_rank();
    constexpr int WARPS = THREADS / 32, U = 4;
    pdl_wait();
    pdl_launch();
    const int n_free = free_count(c);
    find_first<THREADS>(c, b.first, seqs, n);
    for (int i = threadIdx.x; i < n; i += THREADS) {
        int s = entry_seq(c, seqs, i);
        b.cols[i] = 0;
        if (s >= 0 && b.first[s] != i) {
            atomicOr(c.status, PROX_CACHE_BAD_SEQ);
            s = -1;
        }
        if (s >= 0) b.cols[i] = seq_state(c, s).held;
        b.seq[i] = s;
    }
    if (threadIdx.x == 0) b.odd = 0;
    __syncthreads();
    const int chunks = sum_chunks<THREADS>(b, n);
    const int ctas = cl.num_blocks(), per = (chunks + ctas - 1) / ctas;
    const int q0 = min(rank * per, chunks), q1 = min(q0 + per, chunks);
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const bool kept = q1 - q0 <= kWindow;
    for (int q = q0 + threadIdx.x; kept && q < q1; q += THREADS)
        w.owner[q - q0] = (uint16_t)find_entry(b.chunk, n, q);
    __syncthreads();
    auto page_at = [&](int q) {  // this lane's page of chunk q, -1 = none
        if (q >= q1) return -1;
        const int i = kept ? w.owner[q - q0] : find_entry(b.chunk, n, q);
        const int j = (q - b.chunk[i]) * 32 + lane;
        if (j >= b.cols[i]) return -1;
        const int p = c.page_table[(size_t)b.seq[i] * c.max_pages + j];
        if (page_ok(c, p)) return p;
        atomicOr(c.status, PROX_CACHE_BAD_STATE);
        return -1;
    };
    // the CTA's pages, U chunks a warp in flight; f(chunk, page of this lane or -1)
    auto each = [&](int from, int to, auto f) {
        for (int q = from + wid; q < to; q += WARPS * U) {
            int p[U];
#pragma unroll
            for (int u = 0; u < U; ++u) p[u] = q + u * WARPS < to ? page_at(q + u * WARPS) : -1;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (q + u * WARPS < to) f(q + u * WARPS, p[u]);
        }
    };
    each(q0, q1, [&](int, int p) {
        // a count that was 0 or less belongs to a page that is free already
        if (p >= 0 && atomicSub(&c.ref_count[p], 1) <= 0) {
            atomicOr(c.status, PROX_CACHE_BAD_STATE);
            b.odd = 1;
        }
    });
    __threadfence();
    cl.sync();
    each(q0, q1, [&](int q, int p) {
        if (p < 0) return;
        const int r = __ldcg(&c.ref_count[p]);
        if (r == 0 || r < kClaimEnd) atomicMin(&c.ref_count[p], kClaim + q * 32 + lane);
    });
    __threadfence();
    cl.sync();
    // pages this CTA pushes; their masks stay if all of its chunks are kept
    if (threadIdx.x == 0) b.count = 0;
    __syncthreads();
    int mine = 0;
    each(q0, q1, [&](int q, int p) {
        const bool won = p >= 0 && __ldcg(&c.ref_count[p]) == kClaim + q * 32 + lane;
        const unsigned m = __ballot_sync(0xffffffffu, won);
        mine += __popc(m);
        if (kept && lane == 0) w.mask[q - q0] = m;
    });
    if (lane == 0 && mine) atomicAdd(&b.count, mine);
    cl.sync();
    int at = n_free, all = n_free;
    for (int r = 0; r < ctas; ++r) {
        const int k = *cl.map_shared_rank(&b.count, r);
        if (r < rank) at += k;
        all += k;
    }
    for (int from = q0; from < q1; from += kWindow) {
        const int to = min(from + kWindow, q1);
        if (!kept) {
            each(from, to, [&](int q, int p) {
                const bool won = p >= 0 && __ldcg(&c.ref_count[p]) == kClaim + q * 32 + lane;
                const unsigned m = __ballot_sync(0xffffffffu, won);
                if (lane == 0) w.mask[q - from] = m;
            });
            __syncthreads();
        }
        // places of the window's chunks: each thread sums a run of them
        const int run = (to - from + THREADS - 1) / THREADS, k0 = threadIdx.x * run;
        int sum = 0, total;
        for (int k = 0; k < run && from + k0 + k < to; ++k) sum += __popc(w.mask[k0 + k]);
        int place = at + block_scan<THREADS>(sum, b.tmp, &total);
        for (int k = 0; k < run && from + k0 + k < to; ++k) {
            w.before[k0 + k] = place;
            place += __popc(w.mask[k0 + k]);
        }
        __syncthreads();
        each(from, to, [&](int q, int p) {
            const unsigned m = w.mask[q - from];
            if (!(m >> lane & 1)) return;
            const int pos = w.before[q - from] + __popc(m & ((1u << lane) - 1));
            if (pos < c.n_pages) c.free_list[pos] = p;
            c.ref_count[p] = 0;
        });
        at += total;
        __syncthreads();
    }
    cl.sync();  // remote counts are read, codes are gone
    // counts that a page listed too often left below 0
    if (b.odd) each(q0, q1, [&](int, int p) {
        if (p >= 0 && __ldcg(&c.ref_count[p]) < 0) atomicMax(&c.ref_count[p], 0);
    });
    if (rank == 0) {
        if (threadIdx.x == 0) *c.n_free = min(all, c.n_pages);
        for (int i = threadIdx.x; i < n; i += THREADS)
            if (b.seq[i] >= 0) c.length[b.seq[i]] = c.held[b.seq[i]] = 0;
    }
}

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------
// one CTA a row; its threads move the row's 16-byte pieces of k and v. A call is a
// chain of reads (offsets, sequence, length, page, and the row beside them): 4 us.
__global__ void __launch_bounds__(256)
    k_cache_append(const prox_cache c, int layer, int n, const int32_t *seqs, const int32_t *cu,
                   const uint16_t *k, int64_t k_stride, const uint16_t *v, int64_t v_stride) {
    pdl_wait();
    pdl_launch();
    const int row = blockIdx.x, lane = threadIdx.x & 31;
    // the row itself is on its way while its place is looked up
    const int per = c.head_dim / 8, pieces = c.n_kv_heads * per;
    const uint4 *kr = reinterpret_cast<const uint4 *>(k + row * k_stride);
    const uint4 *vr = reinterpret_cast<const uint4 *>(v + row * v_stride);
    uint4 head = make_uint4(0, 0, 0, 0);
    if ((int)threadIdx.x < 2 * pieces)
        head = (int)threadIdx.x < pieces ? kr[threadIdx.x] : vr[threadIdx.x - pieces];
    // entry of the row: the number of ends at or before it. Lanes keep what they
    // read of their entry, so that up to 32 entries need one round of reads.
    int e = 0, start = 0, seq = -1;
    for (int b = 0; b < n; b += 32) {
        const int i = b + lane;
        const int lo = i < n ? cu[i] : 0, hi = i < n ? cu[i + 1] : 0, q = i < n ? seqs[i] : -1;
        const int k = __popc(__ballot_sync(0xffffffffu, i < n && hi <= row));
        e += k;
        if (k < 32 && e < n && e < b + 32) {
            start = __shfl_sync(0xffffffffu, lo, k);
            seq = __shfl_sync(0xffffffffu, q, k);
            break;
        }
    }
    if (e >= n) return;  // behind the last sequence
    const int t = row - start, s = seq;
    if (s < 0 || s >= c.max_seqs) {
        if (s != -1 && threadIdx.x == 0) atomicOr(c.status, PROX_CACHE_BAD_SEQ);
        return;
    }
    const SeqState st = seq_state(c, s);
    bool twice = false;
    for (int b = 0; b < e; b += 32) {
        const int i = b + lane;
        twice |= __any_sync(0xffffffffu, i < e && seqs[i] == s && cu[i + 1] > cu[i]);
    }
    const long pos = (long)st.len + t;
    if (twice || t < 0 || pos >= (long)st.held * c.page_size) {
        if (threadIdx.x == 0)
            atomicOr(c.status, twice ? PROX_CACHE_BAD_SEQ
                                     : t < 0 ? PROX_CACHE_BAD_ARG : PROX_CACHE_FULL);
        return;
    }
    const int page = c.page_table[(size_t)s * c.max_pages + pos / c.page_size];
    if (!page_ok(c, page)) {
        if (threadIdx.x == 0) atomicOr(c.status, PROX_CACHE_BAD_STATE);
        return;
    }
    const size_t at = ((size_t)layer * c.n_pages + page) * c.n_kv_heads * c.page_size +
                      (size_t)(pos % c.page_size);
    for (int i = threadIdx.x; i < 2 * pieces; i += blockDim.x) {
        const int which = i >= pieces, p = i - which * pieces;
        const int h = p / per, d = p - h * per;
        const uint4 x = i == (int)threadIdx.x ? head : which ? vr[p] : kr[p];
        *reinterpret_cast<uint4 *>((which ? c.v : c.k) +
                                   (at + (size_t)h * c.page_size) * c.head_dim + d * 8) = x;
    }
}

// ---------------------------------------------------------------------------
// compact
// ---------------------------------------------------------------------------
// checks entry i (whole CTA): its sequence, or -1; rows kept in *count
__device__ int check_path(const prox_cache &c, int n, const int32_t *seqs, const int32_t *path,
                          int max_path, const int32_t *n_path, int i, SeqState *st, int *count,
                          bool flag) {
    const int s = seqs[i];
    bool twice = false;
    if (s < 0 || s >= c.max_seqs) {
        if (flag && s != -1 && threadIdx.x == 0) atomicOr(c.status, PROX_CACHE_BAD_SEQ);
        return -1;
    }
    for (int j = threadIdx.x; j < i; j += blockDim.x) twice |= seqs[j] == s;
    twice = __syncthreads_or(twice);
    if (twice) {
        if (flag && threadIdx.x == 0) atomicOr(c.status, PROX_CACHE_BAD_SEQ);
        return -1;
    }
    *st = seq_state(c, s);
    const int m = n_path[i], room = st->held * c.page_size - st->len;
    bool bad = m < 0 || m > max_path;
    for (int j = threadIdx.x; !bad && j < m; j += blockDim.x) {
        const int p = path[(size_t)i * max_path + j];
        bad |= p < 0 || p >= room || (j > 0 && path[(size_t)i * max_path + j - 1] >= p);
    }
    bad = __syncthreads_or(bad);
    if (bad) {
        if (flag && threadIdx.x == 0) atomicOr(c.status, PROX_CACHE_BAD_ARG);
        return -1;
    }
    const int32_t *table = c.page_table + (size_t)s * c.max_pages;
    for (int j = threadIdx.x; j < m; j += blockDim.x)
        bad |= !page_ok(c, table[(st->len + path[(size_t)i * max_path + j]) / c.page_size]) ||
               !page_ok(c, table[(st->len + j) / c.page_size]);
    bad = __syncthreads_or(bad);
    if (bad) {
        if (flag && threadIdx.x == 0) atomicOr(c.status, PROX_CACHE_BAD_STATE);
        return -1;
    }
    *count = m;
    return s;
}

// One CTA handles some of an entry's (layer, k or v, head) rows; a group of
// head_dim / 8 lanes follows the path for one of them, 16 bytes a lane. Paths
// ascend, so a row is read (eight ahead) before anything is written over it.
__global__ void __launch_bounds__(256)
    k_cache_compact(const prox_cache c, int n, const int32_t *seqs, const int32_t *path,
                    int max_path, const int32_t *n_path) {
    pdl_wait();
    pdl_launch();
    __shared__ int s_from[kMaxPath], s_to[kMaxPath];   // page row (page * page_size + offset), -1
    const int i = blockIdx.x;
    SeqState st;
    int m = 0;
    const int s = check_path(c, n, seqs, path, max_path, n_path, i, &st, &m, blockIdx.y == 0);
    if (s < 0 || m == 0) return;
    const int32_t *table = c.page_table + (size_t)s * c.max_pages;
    const int ps = c.page_size;
    for (int j = threadIdx.x; j < m; j += blockDim.x) {
        const int a = st.len + path[(size_t)i * max_path + j], b = st.len + j;
        const int pa = table[a / ps], pb = table[b / ps];
        // (n_pages * page_size fits in 31 bits)
        s_from[j] = a != b ? pa * ps + a % ps : -1;
        s_to[j] = pb * ps + b % ps;
    }
    __syncthreads();
    const int lanes = c.head_dim / 8;                  // 8 or 16
    const int groups = blockDim.x / lanes, g = threadIdx.x / lanes, piece = threadIdx.x % lanes;
    const int items = c.n_layers * 2 * c.n_kv_heads;
    for (int it = blockIdx.y * groups + g; it < items; it += gridDim.y * groups) {
        const int h = it % c.n_kv_heads, r = it / c.n_kv_heads;
        const int layer = r >> 1;
        uint4 *pool = reinterpret_cast<uint4 *>(r & 1 ? c.v : c.k) +
                      (size_t)layer * c.n_pages * c.n_kv_heads * ps * lanes;
        auto place = [&](int pr) {
            return pool + (((size_t)(pr / ps) * c.n_kv_heads + h) * ps + pr % ps) * lanes + piece;
        };
        for (int j = 0; j < m; j += 8) {
            uint4 v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (j + u < m && s_from[j + u] >= 0) v[u] = *place(s_from[j + u]);
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (j + u < m && s_from[j + u] >= 0) *place(s_to[j + u]) = v[u];
        }
    }
}

__global__ void __launch_bounds__(256)
    k_cache_commit(const prox_cache c, int n, const int32_t *seqs, const int32_t *path,
                   int max_path, const int32_t *n_path, uint8_t *ok_out) {
    const int i = blockIdx.x;
    SeqState st;
    int m = 0;
    // (what is checked was there before the kernel that moves the rows let this
    // one start, and is not changed by it)
    const int s = check_path(c, n, seqs, path, max_path, n_path, i, &st, &m, false);
    pdl_wait();
    pdl_launch();
    if (threadIdx.x == 0) {
        if (s >= 0 && m > 0) c.length[s] = st.len + m;
        if (ok_out) ok_out[i] = s >= 0 ? 1 : 0;
    }
}

template <typename... P, typename... A>
cudaError_t launch(void (*kern)(P...), dim3 grid, int block, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (smem) {
        cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void *>(kern), smem);
        if (e != cudaSuccess) return e;
    }
    return cudaLaunchKernelEx(&cfg, kern, P(args)...);
}

// whether the device has a place for the kernel's cluster of more than 8 CTAs,
// which needs as many free SMs side by side (asked once per device and kernel)
bool wide_cluster_fits(const void *f, const cudaLaunchConfig_t &cfg) {
    struct Known {
        const void *f;
        int dev;
        bool fits;
    };
    static Known known[256];
    static int n_known = 0;
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    std::lock_guard<std::mutex> lk(mu);
    int at = 0;
    while (at < n_known && (known[at].f != f || known[at].dev != dev)) ++at;
    bool fits;
    if (at < n_known) {
        fits = known[at].fits;
    } else {
        int clusters = 0;
        fits = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
               cudaOccupancyMaxActiveClusters(&clusters, f, &cfg) == cudaSuccess && clusters > 0;
        if (!fits) cudaGetLastError();
        if (n_known < 256) known[n_known++] = {f, dev, fits};
    }
    return fits;
}

// a bookkeeping kernel on one cluster
template <typename... P, typename... A>
cudaError_t book(void (*kern)(P...), int ctas, int block, size_t smem, cudaStream_t s, A... args) {
    const void *f = reinterpret_cast<const void *>(kern);
    cudaError_t e = set_max_dynamic_smem(f, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (ctas > 8 && !wide_cluster_fits(f, cfg)) {
        cfg.gridDim = dim3(8);
        attr[1].val.clusterDim.x = 8;
    }
    return cudaLaunchKernelEx(&cfg, kern, P(args)...);
}

// the kernel's shape for n entries of cache c (see kFew)
#define BOOK(kern, more, c, n, ...)                                                               \
    ((n) <= kFewEntries && (long)(n) * (c).max_pages <= kFewPages                                  \
         ? book(kern<256, kFew>, kFewCtas, 256, sizeof(Book<kFew>) + (more), s, c, n, __VA_ARGS__) \
     : (n) <= kSome                                                                               \
         ? book(kern<1024, kSome>, kCtas, 1024, sizeof(Book<kSome>) + (more), s, c, n, __VA_ARGS__) \
         : book(kern<1024, kMaxSeqs>, kCtas, 1024, sizeof(Book<kMaxSeqs>) + (more), s, c, n,      \
                __VA_ARGS__))

}  // namespace

cudaError_t launch_cache_init(const prox_cache &c, cudaStream_t s) {
    return launch(k_cache_init, dim3(64), 256, 0, s, c);
}

cudaError_t launch_cache_clear(const prox_cache &c, uint32_t bits, cudaStream_t s) {
    return launch(k_cache_clear, dim3(1), 1, 0, s, c, bits);
}

cudaError_t launch_cache_reserve(const prox_cache &c, int n, const int32_t *seqs,
                                 const int32_t *n_new, uint8_t *ok, cudaStream_t s) {
    return BOOK(k_cache_reserve, 0, c, n, seqs, n_new, ok);
}

cudaError_t launch_cache_append(const prox_cache &c, int layer, int n, const int32_t *seqs,
                                const int32_t *cu, int rows, const uint16_t *k, int64_t k_stride,
                                const uint16_t *v, int64_t v_stride, cudaStream_t s) {
    return launch(k_cache_append, dim3(rows), 256, 0, s, c, layer, n, seqs, cu, k, k_stride, v,
                  v_stride);
}

cudaError_t launch_cache_fork(const prox_cache &c, int n, const int32_t *src, const int32_t *dst,
                              int share, uint8_t *ok, int32_t *ws, int sms, cudaStream_t s) {
    cudaError_t e = BOOK(k_cache_fork, 0, c, n, src, dst, share, ok, ws);
    if (e != cudaSuccess) return e;
    return launch(k_cache_copy, dim3(sms * 4), 256, 0, s, c, (const int32_t *)ws);
}

cudaError_t launch_cache_compact(const prox_cache &c, int n, const int32_t *seqs,
                                 const int32_t *path, int max_path, const int32_t *n_path,
                                 uint8_t *ok, cudaStream_t s) {
    const int groups = 256 / (c.head_dim / 8);
    const long items = (long)c.n_layers * 2 * c.n_kv_heads;
    const int gy = (int)min((items + groups - 1) / groups, 1024L);
    cudaError_t e = launch(k_cache_compact, dim3(n, gy), 256, 0, s, c, n, seqs, path, max_path,
                           n_path);
    if (e != cudaSuccess) return e;
    return launch(k_cache_commit, dim3(n), 256, 0, s, c, n, seqs, path, max_path, n_path, ok);
}

cudaError_t launch_cache_free(const prox_cache &c, int n, const int32_t *seqs, cudaStream_t s) {
    return BOOK(k_cache_free, 16 + sizeof(Window), c, n, seqs);
}

}  // namespace prox
