// Page operations of the paged key/value cache (include/prox_decode.h).
//
// Bookkeeping (reserve, fork, free) runs in one cluster of eight CTAs: the
// entries' page counts are prefix-summed by every CTA for itself, so each
// entry's place on the free list is known without atomics and the result does
// not depend on timing, and the pages are then handled in chunks of 32 columns
// dealt out to the cluster's warps. Decisions are taken from the state before
// the call; a cluster barrier separates these reads from the first write.
// The rows themselves are moved by kernels over the whole GPU (fork's copies,
// append, compact), a warp or a group of lanes per run of rows.
#include "decode_internal.cuh"

#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace cg = cooperative_groups;

namespace prox {
namespace {

constexpr int kCl = 8;                 // CTAs of the bookkeeping cluster (portable size)
constexpr int kBkThreads = 1024;
constexpr int kBkWarps = kBkThreads / 32;
constexpr int kPerThread = kMaxSeqs / kBkThreads;

// exclusive prefix sum over the block (and the total), v per thread
template <typename T>
__device__ T block_scan(T v, T *tmp, T *total) {
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
    if (wid == 0) {
        T w = tmp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const T y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        tmp[lane] = w;
    }
    __syncthreads();
    const T base = wid ? tmp[wid - 1] : T(0);
    *total = tmp[31];
    return base + x - v;
}

// shared memory of a bookkeeping CTA: `first` finds sequences listed twice,
// the others hold what each entry needs
struct Book {
    int first[kMaxSeqs];       // lowest entry that lists the sequence
    int seq[kMaxSeqs];         // sequence of the entry, -1 = left out
    int aux[kMaxSeqs];         // fork: source; reserve: columns held so far
    int cols[kMaxSeqs];        // columns (pages) the entry works on
    int base[kMaxSeqs];        // pages taken by the entries before it
    int chunk[kMaxSeqs + 1];   // chunks of 32 columns before it
    int tmp[32];
    long long wide[32];
    int count;                 // free: pages given back by this CTA
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
__device__ void find_first(const prox_cache &c, Book &b, const int32_t *seqs, int n) {
    for (int s = threadIdx.x; s < c.max_seqs; s += kBkThreads) b.first[s] = 0x7fffffff;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kBkThreads) {
        const int s = seqs[i];
        if (s >= 0 && s < c.max_seqs) atomicMin(&b.first[s], i);
    }
    __syncthreads();
}

// exclusive sums of chunks of 32 columns over the entries; returns their count
__device__ int sum_chunks(Book &b, int n) {
    const int i0 = threadIdx.x * kPerThread;
    int mine = 0, total;
    for (int k = 0; k < kPerThread; ++k)
        if (i0 + k < n) mine += (b.cols[i0 + k] + 31) >> 5;
    int at = block_scan(mine, b.tmp, &total);
    for (int k = 0; k < kPerThread; ++k)
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
template <typename F>
__device__ int take_pages(Book &b, int n, int n_free, uint32_t *status, bool *fits, F need_of) {
    // (sums in 64 bits: refused entries may ask for more pages than there are)
    const int i0 = threadIdx.x * kPerThread;
    int need[kPerThread];
    long long mine = 0, total;
    for (int k = 0; k < kPerThread; ++k) {
        need[k] = i0 + k < n ? need_of(i0 + k) : -1;
        mine += max(need[k], 0);
    }
    long long at = block_scan(mine, b.wide, &total);
    int taken = 0;
    for (int k = 0; k < kPerThread; ++k) {
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
    int best = taken;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) b.tmp[threadIdx.x >> 5] = best;
    __syncthreads();
    best = 0;
    for (int w = 0; w < kBkWarps; ++w) best = max(best, b.tmp[w]);
    __syncthreads();
    return best;
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

// ---------------------------------------------------------------------------
// reserve
// ---------------------------------------------------------------------------
__global__ void __cluster_dims__(kCl, 1, 1) __launch_bounds__(kBkThreads)
    k_cache_reserve(const prox_cache c, int n, const int32_t *seqs, const int32_t *n_new,
                    uint8_t *ok_out) {
    extern __shared__ __align__(16) unsigned char smem[];
    Book &b = *reinterpret_cast<Book *>(smem);
    cg::cluster_group cl = cg::this_cluster();
    const int rank = cl.block_rank();
    pdl_wait();
    pdl_launch();
    const int n_free = free_count(c);
    find_first(c, b, seqs, n);
    bool fits[kPerThread];
    const int taken = take_pages(b, n, n_free, c.status, fits, [&](int i) {
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
    for (int k = 0; k < kPerThread; ++k) {
        const int i = threadIdx.x * kPerThread + k;
        if (i >= n) continue;
        if (!fits[k]) {
            b.seq[i] = -1;
            b.cols[i] = 0;
        }
        if (rank == 0 && ok_out) ok_out[i] = fits[k] ? 1 : 0;
    }
    __syncthreads();
    const int chunks = sum_chunks(b, n);
    cl.sync();  // every CTA has read the state
    const int lane = threadIdx.x & 31;
    for (int q = rank * kBkWarps + (threadIdx.x >> 5); q < chunks; q += kCl * kBkWarps) {
        const int i = find_entry(b.chunk, n, q);
        const int j = (q - b.chunk[i]) * 32 + lane;
        if (j >= b.cols[i]) continue;
        c.page_table[(size_t)b.seq[i] * c.max_pages + b.aux[i] + j] =
            pop_page(c, n_free, b.base[i] + j);
    }
    if (rank == 0) {
        for (int i = threadIdx.x; i < n; i += kBkThreads)
            if (b.seq[i] >= 0 && b.cols[i] > 0) c.held[b.seq[i]] = b.aux[i] + b.cols[i];
        if (threadIdx.x == 0) *c.n_free = n_free - taken;
    }
}

// ---------------------------------------------------------------------------
// fork
// ---------------------------------------------------------------------------
// ws: [0] = page copies, then {source page, target page, rows, -} for each
__global__ void __cluster_dims__(kCl, 1, 1) __launch_bounds__(kBkThreads)
    k_cache_fork(const prox_cache c, int n, const int32_t *src, const int32_t *dst, int share,
                 uint8_t *ok_out, int32_t *ws) {
    extern __shared__ __align__(16) unsigned char smem[];
    Book &b = *reinterpret_cast<Book *>(smem);
    cg::cluster_group cl = cg::this_cluster();
    const int rank = cl.block_rank(), ps = c.page_size;
    pdl_wait();
    pdl_launch();
    const int n_free = free_count(c);
    find_first(c, b, dst, n);
    bool fits[kPerThread];
    int len[kPerThread];
    const int taken = take_pages(b, n, n_free, c.status, fits, [&](int i) {
        const int k = i - threadIdx.x * kPerThread;
        const int d = entry_seq(c, dst, i), s = entry_seq(c, src, i);
        b.seq[i] = -1;
        b.cols[i] = 0;
        if (d < 0) return -1;
        if (b.first[d] != i) {
            atomicOr(c.status, PROX_CACHE_BAD_SEQ);
            return -1;
        }
        if (s < 0) return -1;
        if (c.length[d] != 0 || c.held[d] != 0) {
            atomicOr(c.status, PROX_CACHE_BAD_ARG);
            return -1;
        }
        len[k] = seq_state(c, s).len;
        b.seq[i] = d;
        b.aux[i] = s;
        b.cols[i] = (len[k] + ps - 1) / ps;
        return share ? (len[k] % ps ? 1 : 0) : b.cols[i];
    });
    for (int k = 0; k < kPerThread; ++k) {
        const int i = threadIdx.x * kPerThread + k;
        if (i >= n) continue;
        if (!fits[k]) {
            b.seq[i] = -1;
            b.cols[i] = 0;
        }
        if (rank == 0 && ok_out) ok_out[i] = fits[k] ? 1 : 0;
    }
    __syncthreads();
    const int chunks = sum_chunks(b, n);
    cl.sync();  // every CTA has read the state
    const int lane = threadIdx.x & 31;
    for (int q = rank * kBkWarps + (threadIdx.x >> 5); q < chunks; q += kCl * kBkWarps) {
        const int i = find_entry(b.chunk, n, q);
        const int j = (q - b.chunk[i]) * 32 + lane;
        if (j >= b.cols[i]) continue;
        const int l = min(max(c.length[b.aux[i]], 0), b.cols[i] * ps);
        const int rows = min(ps, l - j * ps);
        int p = c.page_table[(size_t)b.aux[i] * c.max_pages + j];
        const bool good = page_ok(c, p);
        if (!good) atomicOr(c.status, PROX_CACHE_BAD_STATE);
        if (share && rows == ps) {
            if (good) atomicAdd(&c.ref_count[p], 1);
        } else {
            const int k = b.base[i] + (share ? 0 : j);
            const int to = pop_page(c, n_free, k);
            int4 copy = make_int4(p, to, good && to >= 0 ? rows : 0, 0);
            reinterpret_cast<int4 *>(ws + 4)[k] = copy;
            p = to;
        }
        c.page_table[(size_t)b.seq[i] * c.max_pages + j] = p;
    }
    // a target's length is written once its columns are: sources were read above
    // by warps of every CTA, and no target with a length is a source of this call
    cl.sync();
    if (rank == 0) {
        for (int k = 0; k < kPerThread; ++k) {
            const int i = threadIdx.x * kPerThread + k;
            if (i < n && b.seq[i] >= 0) {
                c.length[b.seq[i]] = len[k];
                c.held[b.seq[i]] = b.cols[i];
            }
        }
        if (threadIdx.x == 0) {
            *c.n_free = n_free - taken;
            ws[0] = taken;
        }
    }
}

// rows of the pages of fork's list, all layers: one warp moves the rows of one
// head of one page (contiguous), eight 16-byte pieces a lane in flight
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

__global__ void __cluster_dims__(kCl, 1, 1) __launch_bounds__(kBkThreads)
    k_cache_free(const prox_cache c, int n, const int32_t *seqs) {
    extern __shared__ __align__(16) unsigned char smem[];
    Book &b = *reinterpret_cast<Book *>(smem);
    cg::cluster_group cl = cg::this_cluster();
    const int rank = cl.block_rank();
    pdl_wait();
    pdl_launch();
    const int n_free = free_count(c);
    find_first(c, b, seqs, n);
    for (int i = threadIdx.x; i < n; i += kBkThreads) {
        int s = entry_seq(c, seqs, i);
        b.cols[i] = 0;
        if (s >= 0 && b.first[s] != i) {
            atomicOr(c.status, PROX_CACHE_BAD_SEQ);
            s = -1;
        }
        if (s >= 0) b.cols[i] = seq_state(c, s).held;
        b.seq[i] = s;
    }
    __syncthreads();
    const int chunks = sum_chunks(b, n);
    // each CTA owns a run of chunks, so that pages come out in listing order
    const int per = (chunks + kCl - 1) / kCl;
    const int q0 = min(rank * per, chunks), q1 = min(q0 + per, chunks);
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    auto page_at = [&](int q) {  // this lane's page of chunk q, -1 = none
        if (q >= q1) return -1;
        const int i = find_entry(b.chunk, n, q);
        const int j = (q - b.chunk[i]) * 32 + lane;
        if (j >= b.cols[i]) return -1;
        const int p = c.page_table[(size_t)b.seq[i] * c.max_pages + j];
        if (page_ok(c, p)) return p;
        atomicOr(c.status, PROX_CACHE_BAD_STATE);
        return -1;
    };
    for (int q = q0 + wid; q < q1; q += kBkWarps) {
        const int p = page_at(q);
        // a count that was 0 or less belongs to a page that is free already
        if (p >= 0 && atomicSub(&c.ref_count[p], 1) <= 0) atomicOr(c.status, PROX_CACHE_BAD_STATE);
    }
    __threadfence();
    cl.sync();
    for (int q = q0 + wid; q < q1; q += kBkWarps) {
        const int p = page_at(q);
        if (p < 0) continue;
        const int r = __ldcg(&c.ref_count[p]);
        if (r == 0 || r < kClaimEnd) atomicMin(&c.ref_count[p], kClaim + q * 32 + lane);
    }
    __threadfence();
    cl.sync();
    int mine = 0;
    for (int q = q0 + wid; q < q1; q += kBkWarps) {
        const int p = page_at(q);
        const bool won = p >= 0 && __ldcg(&c.ref_count[p]) == kClaim + q * 32 + lane;
        mine += __popc(__ballot_sync(0xffffffffu, won));
    }
    int total;
    block_scan(lane == 0 ? mine : 0, b.tmp, &total);
    if (threadIdx.x == 0) b.count = total;
    cl.sync();
    int at = n_free, all = n_free;
    for (int r = 0; r < kCl; ++r) {
        const int k = *cl.map_shared_rank(&b.count, r);
        if (r < rank) at += k;
        all += k;
    }
    for (int q = q0; q < q1; q += kBkWarps) {
        const int p = page_at(q + wid);
        const int code = kClaim + (q + wid) * 32 + lane;
        const bool won = p >= 0 && __ldcg(&c.ref_count[p]) == code;
        const unsigned m = __ballot_sync(0xffffffffu, won);
        int sum;
        const int before = block_scan(lane == 0 ? __popc(m) : 0, b.tmp, &sum);
        const int pos = at + __shfl_sync(0xffffffffu, before, 0) + __popc(m & ((1u << lane) - 1));
        if (won) {
            if (pos < c.n_pages) c.free_list[pos] = p;
            c.ref_count[p] = 0;
        }
        at += sum;
    }
    cl.sync();  // remote counts are read, codes are gone
    // counts that a page listed too often left below 0
    for (int q = q0 + wid; q < q1; q += kBkWarps) {
        const int p = page_at(q);
        if (p >= 0 && __ldcg(&c.ref_count[p]) < 0) atomicMax(&c.ref_count[p], 0);
    }
    if (rank == 0) {
        if (threadIdx.x == 0) *c.n_free = min(all, c.n_pages);
    }
    cl.sync();  // every CTA has read lengths and page counts for the last time
    if (rank == 0)
        for (int i = threadIdx.x; i < n; i += kBkThreads)
            if (b.seq[i] >= 0) c.length[b.seq[i]] = c.held[b.seq[i]] = 0;
}

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------
// one CTA a row; its threads move the row's 16-byte pieces of k and v
__global__ void __launch_bounds__(256)
    k_cache_append(const prox_cache c, int layer, int n, const int32_t *seqs, const int32_t *cu,
                   const uint16_t *k, int64_t k_stride, const uint16_t *v, int64_t v_stride) {
    pdl_wait();
    pdl_launch();
    const int row = blockIdx.x, lane = threadIdx.x & 31;
    // entry of the row: the number of ends at or before it
    int e = 0;
    for (int i = lane; i < n + lane; i += 32)
        e += __popc(__ballot_sync(0xffffffffu, i < n && cu[i + 1] <= row));
    if (e >= n) return;  // behind the last sequence
    const int t = row - cu[e];
    const int s = entry_seq(c, seqs, e);
    if (s < 0) return;
    bool twice = false;
    for (int i = lane; i < e + lane; i += 32)
        twice |= __any_sync(0xffffffffu, i < e && seqs[i] == s && cu[i + 1] > cu[i]);
    const SeqState st = seq_state(c, s);
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
    const int per = c.head_dim / 8, pieces = c.n_kv_heads * per;
    const size_t at = ((size_t)layer * c.n_pages + page) * c.n_kv_heads * c.page_size +
                      (size_t)(pos % c.page_size);
    for (int i = threadIdx.x; i < 2 * pieces; i += blockDim.x) {
        const int which = i >= pieces, p = i - which * pieces;
        const int h = p / per, d = p - h * per;
        const uint16_t *from = which ? v + row * v_stride : k + row * k_stride;
        uint16_t *to = which ? c.v : c.k;
        *reinterpret_cast<uint4 *>(to + (at + (size_t)h * c.page_size) * c.head_dim + d * 8) =
            *reinterpret_cast<const uint4 *>(from + (size_t)p * 8);
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
        const bool good = page_ok(c, pa) && page_ok(c, pb);
        if (!good) atomicOr(c.status, PROX_CACHE_BAD_STATE);
        // (n_pages * page_size fits in 31 bits)
        s_from[j] = good && a != b ? pa * ps + a % ps : -1;
        s_to[j] = good ? pb * ps + b % ps : 0;
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
    pdl_wait();
    pdl_launch();
    const int i = blockIdx.x;
    SeqState st;
    int m = 0;
    const int s = check_path(c, n, seqs, path, max_path, n_path, i, &st, &m, false);
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

}  // namespace

cudaError_t launch_cache_init(const prox_cache &c, cudaStream_t s) {
    return launch(k_cache_init, dim3(64), 256, 0, s, c);
}

cudaError_t launch_cache_reserve(const prox_cache &c, int n, const int32_t *seqs,
                                 const int32_t *n_new, uint8_t *ok, cudaStream_t s) {
    return launch(k_cache_reserve, dim3(kCl), kBkThreads, sizeof(Book), s, c, n, seqs, n_new, ok);
}

cudaError_t launch_cache_append(const prox_cache &c, int layer, int n, const int32_t *seqs,
                                const int32_t *cu, int rows, const uint16_t *k, int64_t k_stride,
                                const uint16_t *v, int64_t v_stride, cudaStream_t s) {
    return launch(k_cache_append, dim3(rows), 256, 0, s, c, layer, n, seqs, cu, k, k_stride, v,
                  v_stride);
}

cudaError_t launch_cache_fork(const prox_cache &c, int n, const int32_t *src, const int32_t *dst,
                              int share, uint8_t *ok, int32_t *ws, int sms, cudaStream_t s) {
    cudaError_t e = launch(k_cache_fork, dim3(kCl), kBkThreads, sizeof(Book), s, c, n, src, dst,
                           share, ok, ws);
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
    return launch(k_cache_free, dim3(kCl), kBkThreads, sizeof(Book), s, c, n, seqs);
}

}  // namespace prox
