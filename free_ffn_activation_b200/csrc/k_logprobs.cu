// Log probabilities of given tokens, entropy and top alternatives of rows of
// logits (include/prox_decode.h), in one pass over the logits.
//
// With m the largest logit and z = x - m:
//   log sum exp(x) = m + log s0,           s0 = sum e^z,
//   entropy        = log s0 - s1 / s0,     s1 = sum z e^z,
// so a pass needs a running maximum, s0 and s1, rescaled when the maximum
// grows. The top k come out of the same pass: a logit is looked at again only
// if it is not below the k-th largest found so far.
//
// One row is one CTA, or a cluster of up to eight when there are few rows:
// each CTA takes an equal run of the row's 16-byte vectors, and the first one
// joins the others' sums and candidates through distributed shared memory, so
// no workspace and no second launch is needed, and the result does not depend
// on timing.
//
// Measured on the device: 4,000 rows of 128,257 fp32 with the top 5 (2.05 GB) 319 us in
// short runs, 6.4 TB/s, 98% of the rate of a copy, and 357 to 365 us in long ones (87%),
// which power bounds; 64 rows of 151,936 bf16 with the top 20 17.3 us,
// where the first loads, two selections and the cluster's join outweigh the 3 us of
// reading; one row of 32,000 3.3 us. Sums of two elements an instruction were slower
// (366 against 357 us for the first of these, with 512 threads).
#include "decode_internal.cuh"

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cfloat>
#include <cstdint>

namespace cg = cooperative_groups;

namespace prox {
namespace {

constexpr int kWide = 512, kNarrow = 256;  // threads of a CTA, see narrow_rows
constexpr int kMaxWarps = kWide / 32;
constexpr int kUnroll = 4;          // 16-byte vectors a thread has in flight
constexpr int kMaxTop = 64;
constexpr int kCand = 1024;         // candidates kept between selections
constexpr int kMaxSplit = 8;        // CTAs of a row (portable cluster size)
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// order-preserving code of a float; -0 counts as 0, NaN is above everything
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    if ((u & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    if (k == 0xffffffffu) return __uint_as_float(0x7fc00000u);
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

template <int DT>
struct Elem;
template <>
struct Elem<PROX_FP32> {
    static constexpr int N = 4, BYTES = 4;
    static constexpr uint32_t kLow = 0xff800000u;  // -inf
    static __device__ __forceinline__ float max_of(const uint4 (&v)[kUnroll]) {
        float m = -INFINITY;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            m = max_nan(max_nan(max_nan(__uint_as_float(v[u].x), __uint_as_float(v[u].y)),
                                max_nan(__uint_as_float(v[u].z), __uint_as_float(v[u].w))),
                        m);
        return m;
    }
    static __device__ __forceinline__ void unpack(const uint4 &v, float (&f)[4]) {
        f[0] = __uint_as_float(v.x);
        f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z);
        f[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ float pick(const uint4 &v, int j) {
        return __uint_as_float(j & 2 ? (j & 1 ? v.w : v.z) : (j & 1 ? v.y : v.x));
    }
    static __device__ __forceinline__ float load(const void *p, long i) {
        return static_cast<const float *>(p)[i];
    }
};
template <>
struct Elem<PROX_BF16> {
    static constexpr int N = 8, BYTES = 2;
    static constexpr uint32_t kLow = 0xff80ff80u;  // -inf
    static __device__ __forceinline__ float max_of(const uint4 (&v)[kUnroll]) {
        using P = __nv_bfloat162;  // two elements a comparison; NaN if either is
        auto at = [](uint32_t w) { return *reinterpret_cast<const P *>(&w); };
        P m = __hmax2_nan(__hmax2_nan(at(v[0].x), at(v[0].y)), __hmax2_nan(at(v[0].z), at(v[0].w)));
#pragma unroll
        for (int u = 1; u < kUnroll; ++u)
            m = __hmax2_nan(m, __hmax2_nan(__hmax2_nan(at(v[u].x), at(v[u].y)),
                                           __hmax2_nan(at(v[u].z), at(v[u].w))));
        const float2 f = __bfloat1622float2(m);
        return max_nan(f.x, f.y);
    }
    static __device__ __forceinline__ void unpack(const uint4 &v, float (&f)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            f[2 * k] = bf16lo(w[k]);
            f[2 * k + 1] = bf16hi(w[k]);
        }
    }
    static __device__ __forceinline__ float pick(const uint4 &v, int j) {
        const uint32_t w = j & 4 ? (j & 2 ? v.w : v.z) : (j & 2 ? v.y : v.x);
        return j & 1 ? bf16hi(w) : bf16lo(w);
    }
    static __device__ __forceinline__ float load(const void *p, long i) {
        return __uint_as_float((uint32_t) static_cast<const uint16_t *>(p)[i] << 16);
    }
};
template <>
struct Elem<PROX_FP16> {
    static constexpr int N = 8, BYTES = 2;
    static constexpr uint32_t kLow = 0xfc00fc00u;  // -inf
    static __device__ __forceinline__ float max_of(const uint4 (&v)[kUnroll]) {
        using P = __half2;  // two elements a comparison; NaN if either is
        auto at = [](uint32_t w) { return *reinterpret_cast<const P *>(&w); };
        P m = __hmax2_nan(__hmax2_nan(at(v[0].x), at(v[0].y)), __hmax2_nan(at(v[0].z), at(v[0].w)));
#pragma unroll
        for (int u = 1; u < kUnroll; ++u)
            m = __hmax2_nan(m, __hmax2_nan(__hmax2_nan(at(v[u].x), at(v[u].y)),
                                           __hmax2_nan(at(v[u].z), at(v[u].w))));
        const float2 f = __half22float2(m);
        return max_nan(f.x, f.y);
    }
    static __device__ __forceinline__ void unpack(const uint4 &v, float (&f)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&w[k]));
            f[2 * k] = p.x;
            f[2 * k + 1] = p.y;
        }
    }
    static __device__ __forceinline__ float pick(const uint4 &v, int j) {
        const uint32_t w = j & 4 ? (j & 2 ? v.w : v.z) : (j & 2 ? v.y : v.x);
        return __half2float(__ushort_as_half((unsigned short)(j & 1 ? w >> 16 : w)));
    }
    static __device__ __forceinline__ float load(const void *p, long i) {
        return __half2float(static_cast<const __half *>(p)[i]);
    }
};

// a maximum and the sums that go with it
struct Part {
    float m;
    double s0, s1;
};
// the parts of the warp's first N lanes as one, in a fixed order (in lane 0)
template <int N>
__device__ __forceinline__ Part join_parts(Part p) {
    float M = p.m;
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) M = max_nan(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float z = max_nan((p.m - M) * kLog2e, -1e30f);
    const double r = (double)ex2(z);
    p.s1 = r * (p.s1 + (double)z * p.s0);
    p.s0 = r * p.s0;
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) {
        p.s0 += __shfl_xor_sync(0xffffffffu, p.s0, o);
        p.s1 += __shfl_xor_sync(0xffffffffu, p.s1, o);
    }
    p.m = M;
    return p;
}

struct Shared {
    alignas(16) unsigned long long cand[kCand + 8];  // key << 32 | ~index
    alignas(16) unsigned long long joined[kMaxSplit * kMaxTop + 8];  // all CTAs' (first CTA)
    unsigned long long best[kMaxTop];                // the CTA's top k, descending
    unsigned long long sorted[kMaxTop];
    float m[kMaxWarps];
    double s0[kMaxWarps], s1[kMaxWarps];
    Part cta;                                        // the CTA's sums, read by the first one
    uint32_t warp_key[kMaxWarps];
    int n_cand, n_best;
    int lost;                                        // candidates did not fit
    unsigned long long floor;                        // k-th largest so far (0 = none yet)
    float lse_m;
    double log_s0;
};

// places of `count` distinct codes in descending order: the first `keep` go to
// out. `in` has room for 8 codes more, which are cleared here (0 is no code).
// All threads; starts with a barrier.
template <int THREADS>
__device__ __forceinline__ void select_top(unsigned long long *in, int count, int keep,
                                           unsigned long long *out) {
    if (threadIdx.x < 8) in[count + threadIdx.x] = 0;
    __syncthreads();
    for (int t = threadIdx.x; t < count; t += THREADS) {
        const unsigned long long mine = in[t];
        int rank = 0;
        for (int i = 0; i < count; i += 8) {
            ulonglong2 v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) v[u] = *reinterpret_cast<const ulonglong2 *>(in + i + 2 * u);
#pragma unroll
            for (int u = 0; u < 4; ++u) rank += (v[u].x > mine) + (v[u].y > mine);
        }
        if (rank < keep) out[rank] = mine;
    }
}

// the candidates gathered so far become the top k of them, and the k-th is the
// new floor (all threads; ends with a barrier)
template <int THREADS>
__device__ void condense(Shared &sh, int k) {
    __syncthreads();
    const int count = min(sh.n_cand, kCand);
    select_top<THREADS>(sh.cand, count, k, sh.best);  // (its barrier: all have read n_cand)
    __syncthreads();
    const int keep = min(count, k);
    if (threadIdx.x < keep) sh.cand[threadIdx.x] = sh.best[threadIdx.x];
    if (threadIdx.x == 0) {
        if (sh.n_cand > kCand) sh.lost = 1;
        sh.n_cand = keep;
        if (keep == k) sh.floor = sh.best[k - 1];
    }
    __syncthreads();
}

template <int DT, bool TOP, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) k_logprobs(const LogprobArgs a, int split) {
    using E = Elem<DT>;
    constexpr int N = E::N, WARPS = THREADS / 32;
    __shared__ Shared sh;
    cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int rank = blockIdx.x % split;
    const long row = blockIdx.x / split;
    pdl_wait();
    pdl_launch();
    const unsigned char *base =
        static_cast<const unsigned char *>(a.logits) + row * a.stride * E::BYTES;
    // 16-byte vector v covers the row's elements v * N - off .. + N - 1; those
    // that lie in the row as a whole are dealt out, the rest (fewer than 2 N
    // elements at the row's ends) goes to the first CTA's first threads
    const int off = (int)((reinterpret_cast<uintptr_t>(base) & 15u) / E::BYTES);
    const uint4 *vec = reinterpret_cast<const uint4 *>(base - off * E::BYTES);
    const int first = off ? 1 : 0, last = (int)(((long)a.vocab + off) / N);
    const int nvec = max(last - first, 0), per = (nvec + split - 1) / split;
    const int v0 = first + min(rank * per, nvec), v1 = first + min((rank + 1) * per, nvec);
    const int k = a.top_k;

    // the given tokens' logits are on their way meanwhile (one a thread; more
    // than that are read at the end)
    float given = __uint_as_float(0x7fc00000u);
    if (rank == 0 && tid < a.n_tok) {
        const int t = a.tokens[row * a.n_tok + tid];
        if (t >= 0 && t < a.vocab) given = E::load(base, t);
    }

    // a finite start, so that z is never inf - inf where nothing was seen yet
    float m = -FLT_MAX, s0 = 0.f, s1 = 0.f;
    // makes vm's maximum the running one (s1 in units of log2)
    auto raise_to = [&](float vm) {
        if (!(vm <= m)) {  // larger, or NaN
            const float nm = max_nan(m, vm);
            const float z = (m - nm) * kLog2e, r = ex2(z);
            // s1 holds sum z e^z for the old m: shift every z by m - nm
            s1 = r * fmaf(max_nan(z, -1e30f), s0, s1);
            s0 *= r;
            m = nm;
        }
    };
    auto add = [&](float x) {
        // -inf and far values: e^z is 0, and z e^z must be too
        const float z = max_nan((x - m) * kLog2e, -1e30f);
        const float e = ex2(z);
        s0 += e;
        s1 = fmaf(e, z, s1);
    };
    auto offer = [&](float x, long i, unsigned long long fl) {
        const unsigned long long code =
            ((unsigned long long)key_of(x) << 32) | (uint32_t)~(uint32_t)i;
        if (code > fl) {  // (the floor itself is in already)
            const int at = atomicAdd(&sh.n_cand, 1);
            if (at < kCand) sh.cand[at] = code;
        }
    };

    if constexpr (TOP) {
        if (tid == 0) {
            sh.n_cand = 0;
            sh.floor = 0;
            sh.lost = 0;
        }
        __syncthreads();
    }
    if (rank == 0 && tid < 2 * N) {
        const long head = min((long)(off ? N - off : 0), (long)a.vocab);
        const long tail = max(head, (long)last * N - off);
        const long i = tid < N ? tid : tail + tid - N;
        if (tid < N ? i < head : i < a.vocab) {
            const float x = E::load(base, i);
            raise_to(x);
            add(x);
            if constexpr (TOP) offer(x, i, 0);
        }
    }

    constexpr int kStep = THREADS * kUnroll;
    uint4 next[kUnroll];
    auto fetch = [&](int v) {  // vectors behind the CTA's last one: -inf
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            next[u] = make_uint4(E::kLow, E::kLow, E::kLow, E::kLow);
            if (v + u * THREADS < v1) next[u] = __ldcs(vec + v + u * THREADS);
        }
    };
    unsigned long long fl = 0;
    float flv = key_value(0);  // NaN: nothing is below it
    int steps = 0, refresh = 1;
    fetch(v0 + tid);
// (two steps unrolled | one, us: 2,000 rows of 151,936 bf16 with the top 20 230 | 206,
// of 32,000 with the top 5 65 | 54; without alternatives 107.8 | 110.6; 128,256 fp32
// with the top 5 170 | 170, without 160.3 | 162.6)
#pragma unroll(TOP && N == 8 ? 1 : 2)
    for (int vb = v0; vb < v1; vb += kStep) {
        const int v = vb + tid;
        uint4 cur[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) cur[u] = next[u];
        if (vb + kStep < v1) fetch(v + kStep);
        const float vmax = E::max_of(cur);
        raise_to(vmax);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            float x[N];
            E::unpack(cur[u], x);
#pragma unroll
            for (int j = 0; j < N; ++j) add(x[j]);
        }
        if constexpr (TOP) {
            if (steps == 0) {
                // A first floor: of W full warps, each has r lanes whose maximum
                // is at least its r-th largest; with r W >= k the smallest of
                // these values has k elements at or above it.
                const int full = min(WARPS, (v1 - v0) / 32);
                const int r = full ? (k + full - 1) / full : 33;
                if (r <= 32) {
                    uint32_t key = key_of(vmax), rth = 0;
                    for (int i = 0; i < r; ++i) {
                        rth = __reduce_max_sync(0xffffffffu, key);
                        const unsigned who = __ballot_sync(0xffffffffu, key == rth);
                        if (lane == __ffs(who) - 1) key = 0;
                    }
                    if (lane == 0) sh.warp_key[wid] = wid < full ? rth : 0xffffffffu;
                    __syncthreads();
                    uint32_t lo = sh.warp_key[lane % WARPS];
                    lo = __reduce_min_sync(0xffffffffu, lo);
                    // below any index: elements of the floor's value are candidates
                    fl = (unsigned long long)lo << 32;
                    flv = key_value(lo);
                }
            }
            if (!(vmax < flv)) {
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    if (v + u * THREADS >= v1) continue;
                    float x[N];
                    E::unpack(cur[u], x);
                    const long i = (long)(v + u * THREADS) * N - off;
                    unsigned hits = 0;
#pragma unroll
                    for (int j = 0; j < N; ++j) hits |= x[j] < flv ? 0u : 1u << j;
                    while (hits) {
                        const int j = __ffs(hits) - 1;
                        hits &= hits - 1;
                        offer(E::pick(cur[u], j), i + j, fl);
                    }
                }
            }
            // the floor is raised after steps 1, 4, 16, ...: of n elements
            // about k ln 4 pass the floor of the first n / 4
            if (++steps == refresh) {
                refresh *= 4;
                condense<THREADS>(sh, k);
                if (sh.floor) {
                    fl = sh.floor;
                    flv = key_value((uint32_t)(fl >> 32));
                }
            }
        }
    }
    if constexpr (TOP) {
        condense<THREADS>(sh, k);
        if (sh.lost) {
            // More candidates at once than there is room for (rising rows): the
            // row is read again, a vector a thread at a time, in rounds that each
            // take what fits and raise the floor. (What was kept is a part of the
            // row; all of it is offered again except what the floor rules out.)
            __syncthreads();
            if (tid == 0) sh.n_cand = 0;
            fl = 0;
            __syncthreads();
            if (rank == 0 && tid < 2 * N) {
                const long head = min((long)(off ? N - off : 0), (long)a.vocab);
                const long tail = max(head, (long)last * N - off);
                const long i = tid < N ? tid : tail + tid - N;
                if (tid < N ? i < head : i < a.vocab) offer(E::load(base, i), i, 0);
            }
            __syncthreads();  // (these are offered once: before the room fills)
            for (int vb = v0; vb < v1; vb += THREADS) {
                const int v = vb + tid;
                unsigned pending = v < v1 ? (1u << N) - 1u : 0u;
                float x[N] = {};
                if (v < v1) E::unpack(vec[v], x);
                for (;;) {
                    bool more = false;
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        if (!(pending >> j & 1)) continue;
                        const unsigned long long code =
                            ((unsigned long long)key_of(x[j]) << 32) |
                            (uint32_t)~(uint32_t)((long)v * N - off + j);
                        const int at = code > fl ? atomicAdd(&sh.n_cand, 1) : 0;
                        if (code > fl && at < kCand) sh.cand[at] = code;
                        if (code <= fl || at < kCand)
                            pending &= ~(1u << j);
                        else
                            more = true;
                    }
                    more = __syncthreads_or(more);
                    if (more || sh.n_cand > kCand / 2) {
                        condense<THREADS>(sh, k);
                        if (sh.n_cand == k) fl = sh.cand[k - 1];
                    }
                    __syncthreads();
                    if (!more) break;
                }
            }
            condense<THREADS>(sh, k);
        }
    }

    // the CTA's sums, in a fixed order
    float wm = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) wm = max_nan(wm, __shfl_xor_sync(0xffffffffu, wm, o));
    {
        const float z = (m - wm) * kLog2e, r = ex2(z);
        double d1 = (double)(r * fmaf(max_nan(z, -1e30f), s0, s1)), d0 = (double)(r * s0);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            d0 += __shfl_xor_sync(0xffffffffu, d0, o);
            d1 += __shfl_xor_sync(0xffffffffu, d1, o);
        }
        if (lane == 0) {
            sh.m[wid] = wm;
            sh.s0[wid] = d0;
            sh.s1[wid] = d1;
        }
    }
    __syncthreads();
    if (wid == 0) {
        const Part p = join_parts<WARPS>({lane < WARPS ? sh.m[lane] : -FLT_MAX,
                                           lane < WARPS ? sh.s0[lane] : 0.0,
                                           lane < WARPS ? sh.s1[lane] : 0.0});
        if (lane == 0) {
            sh.cta = p;
            if (TOP) sh.n_best = sh.n_cand;
        }
    }
    if (split > 1) {
        cl.sync();
        if (rank != 0) {
            cl.sync();  // the first CTA has read this one's memory
            return;
        }
    } else {
        __syncthreads();
    }
    if (TOP && split > 1) {
        // places without a code are 0 and come last
        for (int t = tid; t < split * k; t += THREADS) {
            const int r = t / k, i = t - r * k;
            const Shared *o = cl.map_shared_rank(&sh, r);
            sh.joined[t] = i < o->n_best ? o->best[i] : 0;
        }
    }
    if (wid == 0) {
        Part p = {-FLT_MAX, 0.0, 0.0};
        if (lane < split) p = cl.map_shared_rank(&sh, lane)->cta;
        p = join_parts<kMaxSplit>(p);
        if (lane == 0) {
            const double ls = log(p.s0);
            sh.lse_m = p.m;
            sh.log_s0 = ls;
            if (a.entropy)
                a.entropy[row] = p.s0 == 0 ? 0.f : (float)(ls - 0.6931471805599453 * (p.s1 / p.s0));
        }
    }
    if (TOP && split > 1) {
        __syncthreads();
        select_top<THREADS>(sh.joined, split * k, k, sh.sorted);
    }
    __syncthreads();
    const float M = sh.lse_m;
    const double ls = sh.log_s0;
    // an empty row (every logit -inf) has s0 = 0: every token has logp -inf
    auto logp = [&](float x) {
        return ls == -INFINITY ? -INFINITY : (float)((double)x - (double)M - ls);
    };
    if constexpr (TOP) {
        if (tid < k) {
            const unsigned long long code = split > 1 ? sh.sorted[tid] : sh.best[tid];
            a.top_ids[row * k + tid] = (int32_t)~(uint32_t)code;
            a.top_logp[row * k + tid] = logp(key_value((uint32_t)(code >> 32)));
        }
    }
    // (NaN for a token out of range goes through)
    if (tid < a.n_tok) a.logp[row * a.n_tok + tid] = isnan(given) ? given : logp(given);
    for (int i = tid + THREADS; i < a.n_tok; i += THREADS) {
        const int t = a.tokens[row * a.n_tok + i];
        a.logp[row * a.n_tok + i] =
            t >= 0 && t < a.vocab ? logp(E::load(base, t)) : __uint_as_float(0x7fc00000u);
    }
    if (split > 1) cl.sync();
}

template <int DT, int THREADS>
cudaError_t launch_as(const LogprobArgs &a, int split, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.rows * split));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return a.top_k ? cudaLaunchKernelEx(&cfg, k_logprobs<DT, true, THREADS>, a, split)
                   : cudaLaunchKernelEx(&cfg, k_logprobs<DT, false, THREADS>, a, split);
}
template <int DT>
cudaError_t launch_dt(const LogprobArgs &a, bool narrow, int split, cudaStream_t s) {
    return narrow ? launch_as<DT, kNarrow>(a, split, s) : launch_as<DT, kWide>(a, split, s);
}

// CTAs of 256 threads (four an SM) rather than 512 (two): with many rows the other
// three read on while one is at the barriers of its selections and its row's end, and
// short rows have few steps. Between them a row's selections want the threads. (us;
// 512 | 256 threads)
//   rows    151,936 bf16, top 20   151,936 bf16   128,256 fp32, top 5   32,000 bf16, top 5
//   1           10.6 |  10.8        4.7 |   4.6       9.0 |  10.1           7.2 |  6.6
//   64          17.4 |  20.1        8.8 |   8.3      15.2 |  16.2           9.7 |  7.8
//   600         75.4 |  88.9       45.3 |  44.4      69.4 |  71.1          27.3 | 21.9
//   2,000      206.5 | 203.2      121.1 | 107.7     185.1 | 171.0          71.6 | 52.4
//   4,000 (short runs)                              357   | 319
bool narrow_rows(int rows, int vectors, int sms) { return rows >= 8 * sms || vectors <= 4096; }

}  // namespace

cudaError_t launch_logprobs(const LogprobArgs &a, int dtype, int sms, cudaStream_t s) {
    // CTAs of a row: while the rows alone leave SMs without a CTA, and each
    // CTA keeps a few vectors a thread to read
    const int vectors = a.vocab / (dtype == PROX_FP32 ? 4 : 8);
    const bool narrow = narrow_rows(a.rows, vectors, sms);
    int split = 1;
    while (split < kMaxSplit && (long)a.rows * split * 2 <= 2L * sms &&
           vectors / (split * 2) >= (narrow ? kNarrow : kWide) / 2)
        split *= 2;
    switch (dtype) {
        case PROX_BF16: return launch_dt<PROX_BF16>(a, narrow, split, s);
        case PROX_FP16: return launch_dt<PROX_FP16>(a, narrow, split, s);
        default: return launch_dt<PROX_FP32>(a, narrow, split, s);
    }
}

}  // namespace prox
