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

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
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
    static __device__ __forceinline__ void unpack(const uint4 &v, float (&f)[4]) {
        f[0] = __uint_as_float(v.x);
        f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z);
        f[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ float load(const void *p, long i) {
        return static_cast<const float *>(p)[i];
    }
};
template <>
struct Elem<PROX_BF16> {
    static constexpr int N = 8, BYTES = 2;
    static __device__ __forceinline__ void unpack(const uint4 &v, float (&f)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            f[2 * k] = bf16lo(w[k]);
            f[2 * k + 1] = bf16hi(w[k]);
        }
    }
    static __device__ __forceinline__ float load(const void *p, long i) {
        return __uint_as_float((uint32_t) static_cast<const uint16_t *>(p)[i] << 16);
    }
};
template <>
struct Elem<PROX_FP16> {
    static constexpr int N = 8, BYTES = 2;
    static __device__ __forceinline__ void unpack(const uint4 &v, float (&f)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&w[k]));
            f[2 * k] = p.x;
            f[2 * k + 1] = p.y;
        }
    }
    static __device__ __forceinline__ float load(const void *p, long i) {
        return __half2float(static_cast<const __half *>(p)[i]);
    }
};

struct Shared {
    unsigned long long cand[kCand];                  // key << 32 | ~index
    unsigned long long best[kMaxTop];                // the CTA's top k, descending
    unsigned long long joined[kMaxSplit * kMaxTop];  // all CTAs' (first CTA only)
    unsigned long long sorted[kMaxTop];
    float m[kWarps];
    double s0[kWarps], s1[kWarps];
    float cta_m;                                     // the CTA's sums, read by the first one
    double cta_s0, cta_s1;
    uint32_t warp_key[kWarps];
    int n_cand, n_best;
    unsigned long long floor;                        // k-th largest so far (0 = none yet)
    float lse_m;
    double log_s0;
};

// places of `count` distinct codes in descending order: the first `keep` go to out
__device__ __forceinline__ void select_top(const unsigned long long *in, int count, int keep,
                                           unsigned long long *out) {
    for (int t = threadIdx.x; t < count; t += kThreads) {
        const unsigned long long mine = in[t];
        int rank = 0;
        for (int i = 0; i < count; ++i) rank += in[i] > mine;
        if (rank < keep) out[rank] = mine;
    }
}

// the candidates gathered so far become the top k of them, and the k-th is the
// new floor (all threads; ends with a barrier)
__device__ void condense(Shared &sh, int k) {
    __syncthreads();
    const int count = min(sh.n_cand, kCand);
    select_top(sh.cand, count, k, sh.best);
    __syncthreads();
    const int keep = min(count, k);
    if (threadIdx.x < keep) sh.cand[threadIdx.x] = sh.best[threadIdx.x];
    if (threadIdx.x == 0) {
        sh.n_cand = keep;
        if (keep == k) sh.floor = sh.best[k - 1];
    }
    __syncthreads();
}

template <int DT, bool TOP>
__global__ void __launch_bounds__(kThreads, 2) k_logprobs(const LogprobArgs a, int split) {
    using E = Elem<DT>;
    constexpr int N = E::N;
    __shared__ Shared sh;
    cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int rank = blockIdx.x % split;
    const long row = blockIdx.x / split;
    pdl_wait();
    pdl_launch();
    const unsigned char *base =
        static_cast<const unsigned char *>(a.logits) + row * a.stride * E::BYTES;
    // vector v covers the row's elements v * N - off .. + N - 1; the first and
    // the last one may reach out of the row
    const int off = (int)((reinterpret_cast<uintptr_t>(base) & 15u) / E::BYTES);
    const uint4 *vec = reinterpret_cast<const uint4 *>(base - off * E::BYTES);
    const int nvec = (a.vocab + off + N - 1) / N;
    const int per = (nvec + split - 1) / split;
    const int v0 = min(rank * per, nvec), v1 = min(v0 + per, nvec);
    if (TOP && tid == 0) {
        sh.n_cand = 0;
        sh.floor = 0;
    }

    auto fetch = [&](int v) {
        const long e0 = (long)v * N - off;
        if (e0 >= 0 && e0 + N <= a.vocab) return __ldcs(vec + v);
        float f[N];
        uint4 r;
#pragma unroll
        for (int j = 0; j < N; ++j)
            f[j] = e0 + j >= 0 && e0 + j < a.vocab ? E::load(base, e0 + j) : -INFINITY;
        if constexpr (DT == PROX_FP32) {
            r = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                           __float_as_uint(f[3]));
        } else {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (DT == PROX_BF16) {
                    w[j] = (__float_as_uint(f[2 * j]) >> 16) |
                           (__float_as_uint(f[2 * j + 1]) & 0xffff0000u);
                } else {
                    const __half2 h = __floats2half2_rn(f[2 * j], f[2 * j + 1]);
                    w[j] = *reinterpret_cast<const uint32_t *>(&h);
                }
            }
            r = make_uint4(w[0], w[1], w[2], w[3]);
        }
        return r;
    };

    // a finite start, so that z is never inf - inf where nothing was seen yet
    float m = -FLT_MAX, s0 = 0.f, s1 = 0.f;
    // one vector into the running sums (s1 in units of log2); returns its maximum
    auto take = [&](const float (&x)[N]) {
        float vm = x[0];
#pragma unroll
        for (int j = 1; j < N; ++j) vm = max_nan(vm, x[j]);
        if (!(vm <= m)) {  // larger, or NaN
            const float nm = max_nan(m, vm);
            const float z = (m - nm) * kLog2e, r = ex2(z);
            // s1 holds sum z e^z for the old m: shift every z by m - nm
            s1 = r * fmaf(max_nan(z, -1e30f), s0, s1);
            s0 *= r;
            m = nm;
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            // -inf and far values: e^z is 0, and z e^z must be too
            const float z = max_nan((x[j] - m) * kLog2e, -1e30f);
            const float e = ex2(z);
            s0 += e;
            s1 = fmaf(e, z, s1);
        }
        return vm;
    };

    if constexpr (TOP) __syncthreads();
    const int k = a.top_k;
    uint4 cur[kUnroll];
    const int step = kThreads * kUnroll;
    auto fetch_all = [&](int v) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            cur[u] = v + u * kThreads + tid < v1 ? fetch(v + u * kThreads + tid) : uint4{};
    };
    fetch_all(v0);
    for (int v = v0; v < v1; v += step) {
        uint4 now[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) now[u] = cur[u];
        if (v + step < v1) fetch_all(v + step);
        float vmax[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            vmax[u] = -INFINITY;
            if (v + u * kThreads + tid < v1) {
                float x[N];
                E::unpack(now[u], x);
                vmax[u] = take(x);
            }
        }
        if constexpr (TOP) {
            if (v == v0) {
                // A first floor: of W full warps, each has r lanes whose maximum
                // is at least its r-th largest; with r W >= k the smallest of
                // these values has k elements at or above it.
                const int full = min(kWarps, (v1 - v0) / 32);
                const int r = full ? (k + full - 1) / full : 33;
                uint32_t key = 0;
#pragma unroll
                for (int u = 0; u < kUnroll; ++u)
                    if (v + u * kThreads + tid < v1) key = max(key, key_of(vmax[u]));
                uint32_t rth = 0;
                if (r <= 32) {
                    for (int i = 0; i < r; ++i) {
                        rth = __reduce_max_sync(0xffffffffu, key);
                        const unsigned who = __ballot_sync(0xffffffffu, key == rth);
                        if (lane == __ffs(who) - 1) key = 0;
                    }
                }
                if (lane == 0) sh.warp_key[wid] = wid < full ? rth : 0xffffffffu;
                __syncthreads();
                if (tid == 0 && r <= 32) {
                    uint32_t lo = 0xffffffffu;
                    for (int w = 0; w < kWarps; ++w) lo = min(lo, sh.warp_key[w]);
                    // any index: elements equal to the floor's value stay candidates
                    sh.floor = (unsigned long long)lo << 32;
                }
                __syncthreads();
            }
            // candidates of this step; a step that does not fit is taken in
            // several rounds, each of which raises the floor
            unsigned pending = 0xffffffffu;
            for (;;) {
                const unsigned long long fl = sh.floor;
                const float flv = key_value((uint32_t)(fl >> 32));
                bool more = false;
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    const int vi = v + u * kThreads + tid;
                    // (a floor of 0 is no floor: its value reads as NaN)
                    if (vi >= v1 || vmax[u] < flv) continue;
                    float x[N];
                    E::unpack(now[u], x);
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        const long e = (long)vi * N - off + j;
                        const unsigned bit = 1u << (u * N + j);
                        if (!(pending & bit) || e < 0 || e >= a.vocab) continue;
                        const unsigned long long code =
                            ((unsigned long long)key_of(x[j]) << 32) | (uint32_t)~(uint32_t)e;
                        if (code <= fl) {  // (the floor itself is in already)
                            pending &= ~bit;
                            continue;
                        }
                        const int at = atomicAdd(&sh.n_cand, 1);
                        if (at < kCand) {
                            sh.cand[at] = code;
                            pending &= ~bit;
                        } else {
                            more = true;
                        }
                    }
                }
                more = __syncthreads_or(more);
                if (!more) break;
                condense(sh, k);
            }
            if (sh.n_cand > 2 * k + 128) condense(sh, k);  // (uniform: after the barrier)
            __syncthreads();
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
    if constexpr (TOP) condense(sh, k);
    __syncthreads();
    if (tid == 0) {
        float M = sh.m[0];
        for (int w = 1; w < kWarps; ++w) M = max_nan(M, sh.m[w]);
        double t0 = 0, t1 = 0;
        for (int w = 0; w < kWarps; ++w) {
            const float z = max_nan((sh.m[w] - M) * kLog2e, -1e30f);
            const double r = (double)ex2(z);
            t0 += r * sh.s0[w];
            t1 += r * (sh.s1[w] + (double)z * sh.s0[w]);
        }
        sh.cta_m = M;
        sh.cta_s0 = t0;
        sh.cta_s1 = t1;
        if (TOP) sh.n_best = sh.n_cand;
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
    if (tid == 0) {
        float M = sh.cta_m;
        for (int r = 1; r < split; ++r) M = max_nan(M, *cl.map_shared_rank(&sh.cta_m, r));
        double t0 = 0, t1 = 0;
        for (int r = 0; r < split; ++r) {
            const Shared *o = r ? cl.map_shared_rank(&sh, r) : &sh;
            const float z = max_nan((o->cta_m - M) * kLog2e, -1e30f);
            const double w = (double)ex2(z);
            t0 += w * o->cta_s0;
            t1 += w * (o->cta_s1 + (double)z * o->cta_s0);
        }
        const double ls = log(t0);
        sh.lse_m = M;
        sh.log_s0 = ls;
        if (a.entropy)
            a.entropy[row] = t0 == 0 ? 0.f : (float)(ls - 0.6931471805599453 * (t1 / t0));
    }
    int found = 0;
    if constexpr (TOP) {
        if (split > 1) {
            for (int r = 0; r < split; ++r) {
                const Shared *o = r ? cl.map_shared_rank(&sh, r) : &sh;
                const int c = o->n_best;
                if (tid < c) sh.joined[found + tid] = o->best[tid];
                found += c;
            }
            __syncthreads();
            select_top(sh.joined, found, k, sh.sorted);
        }
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
    for (int i = tid; i < a.n_tok; i += kThreads) {
        const int t = a.tokens[row * a.n_tok + i];
        a.logp[row * a.n_tok + i] =
            t >= 0 && t < a.vocab ? logp(E::load(base, t)) : __uint_as_float(0x7fc00000u);
    }
    if (split > 1) cl.sync();
}

template <int DT>
cudaError_t launch_dt(const LogprobArgs &a, int split, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.rows * split));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return a.top_k ? cudaLaunchKernelEx(&cfg, k_logprobs<DT, true>, a, split)
                   : cudaLaunchKernelEx(&cfg, k_logprobs<DT, false>, a, split);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobArgs &a, int dtype, int sms, cudaStream_t s) {
    // CTAs of a row: while the rows alone leave SMs without a CTA, and each
    // CTA keeps a few vectors a thread to read
    const int per_vec = dtype == PROX_FP32 ? 4 : 8;
    int split = 1;
    while (split < kMaxSplit && (long)a.rows * split * 2 <= 2L * sms &&
           a.vocab / per_vec / (split * 2) >= kThreads / 2)
        split *= 2;
    switch (dtype) {
        case PROX_BF16: return launch_dt<PROX_BF16>(a, split, s);
        case PROX_FP16: return launch_dt<PROX_FP16>(a, split, s);
        default: return launch_dt<PROX_FP32>(a, split, s);
    }
}

}  // namespace prox
