// Log probabilities of given tokens, entropy and alternatives of logits rows, and the gradient to
// the logits (include/specverify_logprobs.h).

#include "specverify_logprobs.h"

#include <cuda_bf16.h>

#include <cfloat>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <type_traits>

namespace svlp {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBatch = 4;        // 16-byte vectors of a thread in flight
constexpr int kMaxV = 1 << 21;
constexpr int kMaxGiven = SV_LOGPROBS_MAX_GIVEN;
constexpr int kMaxTop = SV_LOGPROBS_MAX_TOP;
constexpr int kPairs = kThreads / 2;
constexpr int kCandidates = 1024;
constexpr int kMaxCluster = 8;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The larger; NaN where either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
// A load of what is read once.
__device__ __forceinline__ uint4 ld_stream16(const uint4* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
// The same of memory that this kernel may write.
__device__ __forceinline__ uint4 ld_own16(const uint4* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ int cluster_rank() {
    int r;
    asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ int cluster_size() {
    int r;
    asm volatile("mov.u32 %0, %cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive;\nbarrier.cluster.wait;" ::: "memory");
}
// The same place in the shared memory of CTA k of the cluster.
template <typename P> __device__ __forceinline__ const P* cluster_at(P* p, int k) {
    uint64_t r;
    asm volatile("mapa.u64 %0, %1, %2;" : "=l"(r) : "l"(p), "r"(k));
    return reinterpret_cast<const P*>(r);
}

// ---------------------------------------------------------------- rows

// Elements of a type in 16-byte vectors.
template <typename T> struct Elt;
template <> struct Elt<__nv_bfloat16> {
    static constexpr int kVec = 8;
    static constexpr uint32_t kLowest = 0xff80ff80u;  // -inf in every place of a word
    static __device__ __forceinline__ float get(const __nv_bfloat16* p) {
        return __bfloat162float(*p);
    }
    static __device__ __forceinline__ __nv_bfloat16 from(float x) { return __float2bfloat16_rn(x); }
    static __device__ __forceinline__ void unpack(const uint4& v, float* f) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    // (NaN only where all are)
    static __device__ __forceinline__ float largest(const uint4& v) {
        auto two = [](uint32_t w) { return reinterpret_cast<const __nv_bfloat162&>(w); };
        const __nv_bfloat162 m = __hmax2(__hmax2(two(v.x), two(v.y)), __hmax2(two(v.z), two(v.w)));
        return fmaxf(__low2float(m), __high2float(m));
    }
    static __device__ __forceinline__ uint4 pack(const float* f) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = reinterpret_cast<const uint32_t&>(h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <> struct Elt<float> {
    static constexpr int kVec = 4;
    static constexpr uint32_t kLowest = 0xff800000u;
    static __device__ __forceinline__ float get(const float* p) { return *p; }
    static __device__ __forceinline__ float from(float x) { return x; }
    static __device__ __forceinline__ void unpack(const uint4& v, float* f) {
        f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ float largest(const uint4& v) {
        return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)),
                     fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
    }
    static __device__ __forceinline__ uint4 pack(const float* f) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                          __float_as_uint(f[3]));
    }
};

// A row as 16-byte vectors: it begins `skew` elements behind a 16-byte boundary, so that vector i
// holds elements i * kVec - skew on.  The first and the last vector may be partly outside.
template <typename T> struct Row {
    static constexpr int kVec = Elt<T>::kVec;
    const T* row;
    int V, skew, vectors;
    __device__ __forceinline__ Row(const T* p, int V_) : row(p), V(V_) {
        skew = (int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
        vectors = (V + skew + kVec - 1) / kVec;
    }
    __device__ __forceinline__ bool whole(int i) const {
        return (i > 0 || skew == 0) && (i + 1) * kVec <= V + skew;
    }
    __device__ __forceinline__ const uint4* at(int i) const {
        return reinterpret_cast<const uint4*>(row - skew) + i;
    }
    // Vector i; -inf in places outside of the row.
    __device__ __forceinline__ uint4 load(int i) const {
        if (whole(i)) return ld_stream16(at(i));
        float f[kVec];
#pragma unroll
        for (int q = 0; q < kVec; ++q) {
            const int e = i * kVec + q - skew;
            f[q] = e >= 0 && e < V ? Elt<T>::get(row + e) : -INFINITY;
        }
        return Elt<T>::pack(f);
    }
};

// A number that orders like the float (NaN above or below all); -0 and +0 are one.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
// An element as one number: larger values first, then lower places; 0 is none.
__device__ __forceinline__ uint64_t key_of(float x, int e) {
    return (uint64_t)ordered(x) << 32 | (0xffffffffu - (uint32_t)e);
}
__device__ __forceinline__ int place_of(uint64_t key) {
    return (int)(0xffffffffu - (uint32_t)key);
}

// Maximum m, sum s of 2^((l - m) c) and sum u of 2^((l - m) c) (l - m).  s is NaN where the row is
// bad, but for a row of -inf alone, where m is -inf and s is 0.
struct Stats {
    float m, s, u;
};
__device__ __forceinline__ void add(Stats& a, const Stats& b, float c) {
    const float m = fmaxf(a.m, b.m);
    const float da = a.m == m || a.m == -INFINITY ? 0.0f : a.m - m;
    const float db = b.m == m || b.m == -INFINITY ? 0.0f : b.m - m;
    const float fa = ex2(da * c), fb = ex2(db * c);
    // (a side so far below that nothing of it is left may have da * s = -inf)
    a.u = (fa > 0.0f ? fa * fmaf(da, a.s, a.u) : 0.0f) +
          (fb > 0.0f ? fb * fmaf(db, b.s, b.u) : 0.0f);
    a.s = a.s * fa + b.s * fb;
    a.m = m;
}

// ---------------------------------------------------------------- log probabilities

struct Args {
    const void* logits;
    long long stride;
    const int32_t* tokens;
    float T, c, c_low;  // c + c_low: log2(e) / T
    int V, given, top;
    float* logprobs;
    float* normalizer;
    float* entropy;
    int32_t* top_tokens;
    float* top_logprobs;
    uint32_t* status;
};

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{ .reg .b64 a, b, c; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mov.b64 c, {%6, %7}; "
        "fma.rn.f32x2 a, a, b, c; mov.b64 {%0, %1}, a; }"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{ .reg .b64 a, b; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; "
        "mul.rn.f32x2 a, a, b; mov.b64 {%0, %1}, a; }"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{ .reg .b64 a, b; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; "
        "add.rn.f32x2 a, a, b; mov.b64 {%0, %1}, a; }"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// A cluster of CTAs per row, each with an equal run of its vectors, read once with the running
// maximum and sums of a softmax; joined through distributed shared memory.
//
// Alternatives.  Each thread knows its largest element and the vector that it is in.  Of the
// maxima of pairs of threads the top-th is a bound: as many elements are at or above it, and
// these are in the vectors of the threads whose own maximum reaches it, about as many again.  Only
// those threads' vectors are read a second time (by their warp, from L2), the elements that reach
// the bound are put in order by counting, and rank 0 joins the lists of the cluster's CTAs.
template <typename T, bool ENTROPY, bool TOP>
__global__ void __launch_bounds__(kThreads, 4) lp_kernel(const Args a) {
    using E = Elt<T>;
    constexpr int VW = E::kVec;
    __shared__ Stats s_warp[kWarps], s_stats;
    __shared__ uint64_t s_pair[kPairs], s_top[kMaxTop], s_bound, s_cand[kCandidates];
    __shared__ int s_count;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int G = cluster_size(), rank = cluster_rank(), r = blockIdx.x / G;

    int token = -1;
    if (tid < a.given) token = a.tokens[(long long)r * a.given + tid];
    if (!__syncthreads_or(token != -1)) return;  // (the whole cluster)
    const Row<T> row((const T*)a.logits + r * a.stride, a.V);
    const int i0 = (int)((long long)row.vectors * rank / G);
    const int i1 = (int)((long long)row.vectors * (rank + 1) / G);
    const uint4 none = make_uint4(E::kLowest, E::kLowest, E::kLowest, E::kLowest);

    Stats st = {-INFINITY, 0.0f, 0.0f};
    int best = i0 + tid;  // the vector that holds this thread's first maximum
    uint4 v[kBatch];
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
        const int k = i0 + tid + q * kThreads;
        v[q] = k < i1 ? row.load(k) : none;
    }
    const bool known = token >= 0 && token < a.V;
    const float given = rank == 0 && known ? E::get(row.row + token) : 0.0f;
    for (int i = i0 + tid; i < i1; i += kThreads * kBatch) {
        uint4 next[kBatch];
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            const int k = i + (kBatch + q) * kThreads;
            next[q] = k < i1 ? row.load(k) : none;
        }
        float top[kBatch];
#pragma unroll
        for (int q = 0; q < kBatch; ++q) top[q] = E::largest(v[q]);
        float most = top[0];
#pragma unroll
        for (int q = 1; q < kBatch; ++q) most = fmaxf(most, top[q]);
        if (most > st.m) {
            if (TOP) {
#pragma unroll
                for (int q = kBatch - 1; q >= 0; --q)
                    if (top[q] == most) best = i + q * kThreads;
            }
            add(st, Stats{most, 0.0f, 0.0f}, a.c);
        }
        const float2 less = both(st.m == -INFINITY ? 0.0f : -st.m);
        float2 s = make_float2(0.0f, 0.0f), u = s;
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            float x[VW];
            E::unpack(v[q], x);
#pragma unroll
            for (int e = 0; e < VW; e += 2) {
                float2 d = add2(make_float2(x[e], x[e + 1]), less);
                float2 p = fma2(d, both(a.c_low), mul2(d, both(a.c)));
                p.x = ex2(p.x);
                p.y = ex2(p.y);
                s = add2(s, p);
                if (ENTROPY) {  // (0 times -inf is NaN)
                    d.x = fmaxf(d.x, -FLT_MAX);
                    d.y = fmaxf(d.y, -FLT_MAX);
                    u = fma2(p, d, u);
                }
            }
        }
        st.s += s.x + s.y;
        st.u += u.x + u.y;
#pragma unroll
        for (int q = 0; q < kBatch; ++q) v[q] = next[q];
    }
    const float mine = st.m;
#pragma unroll
    for (int k = 16; k; k >>= 1) {
        Stats o;
        o.m = __shfl_xor_sync(~0u, st.m, k);
        o.s = __shfl_xor_sync(~0u, st.s, k);
        o.u = __shfl_xor_sync(~0u, st.u, k);
        add(st, o, a.c);
    }
    if (lane == 0) s_warp[w] = st;
    uint64_t key = 0;
    if (TOP) {
        // (the last place of the vector: nothing that equals the maximum is left out)
        if (i0 + tid < i1) key = key_of(mine, min(best * VW + VW - 1 - row.skew, a.V - 1));
        const uint64_t other = __shfl_xor_sync(~0u, key, 1);
        if (!(tid & 1)) s_pair[tid >> 1] = key > other ? key : other;
        if (tid < kMaxTop) s_top[tid] = 0;
        if (tid == 0) s_bound = 0, s_count = 0;
    }
    __syncthreads();
    if (tid == kThreads - 1) {
        Stats t = s_warp[0];
        for (int k = 1; k < kWarps; ++k) add(t, s_warp[k], a.c);
        s_stats = t;
    }
    if (TOP) {
        if (tid < kPairs) {
            const uint64_t p = s_pair[tid];
            int above = 0;
#pragma unroll 8
            for (int k = 0; k < kPairs; ++k) above += s_pair[k] > p;
            if (p && above == a.top - 1) s_bound = p;
        }
        __syncthreads();
        const uint64_t bound = s_bound;
        // Vectors of the threads whose maximum reaches the bound.
        const int per = (i1 - i0 + kThreads - 1) / kThreads;
        for (uint32_t reach = __ballot_sync(~0u, key && key >= bound); reach; reach &= reach - 1) {
            const int t = (w << 5) + __ffs(reach) - 1;
            for (int j = lane; j < per; j += 32) {
                const int i = i0 + t + j * kThreads;
                if (i >= i1) continue;
                float x[VW];
                E::unpack(row.load(i), x);
#pragma unroll
                for (int e = 0; e < VW; ++e) {
                    const int at = i * VW + e - row.skew;
                    if (at < 0 || at >= a.V) continue;
                    const uint64_t k = key_of(x[e], at);
                    if (k < bound) continue;
                    const int n = atomicAdd(&s_count, 1);
                    if (n < kCandidates) s_cand[n] = k;
                }
            }
        }
        __syncthreads();
        const int n = s_count;
        if (n <= kCandidates) {
            for (int i = tid; i < n; i += kThreads) {
                const uint64_t k = s_cand[i];
                int above = 0;
                for (int j = 0; j < n; ++j) above += s_cand[j] > k;
                if (above < a.top) s_top[above] = k;
            }
        } else {
            // Large elements that lie together, many more than are wanted: the whole run again for
            // each of them.
            uint64_t last = ~0ull;
            for (int out = 0; out < a.top; ++out) {
                uint64_t most = 0;
                for (int i = i0 + tid; i < i1; i += kThreads) {
                    float x[VW];
                    E::unpack(row.load(i), x);
#pragma unroll
                    for (int e = 0; e < VW; ++e) {
                        const int at = i * VW + e - row.skew;
                        const uint64_t k = at < 0 || at >= a.V ? 0 : key_of(x[e], at);
                        if (k < last && k > most) most = k;
                    }
                }
                for (int k = 16; k; k >>= 1) {
                    const uint64_t o = __shfl_xor_sync(~0u, most, k);
                    most = o > most ? o : most;
                }
                if (lane == 0) s_pair[w] = most;
                __syncthreads();
                for (int k = 0; k < kWarps; ++k) most = s_pair[k] > most ? s_pair[k] : most;
                if (tid == 0) s_top[out] = most;
                last = most;
                __syncthreads();
            }
        }
    }
    cluster_sync();
    if (rank == 0) {
        Stats t = s_stats;
        for (int k = 1; k < G; ++k) add(t, *cluster_at(&s_stats, k), a.c);
        const bool bad = !(t.s > 0.0f && t.s < INFINITY) || t.m == INFINITY;
        const float log_s = bad ? NAN : logf(t.s), m = bad ? NAN : t.m;
        if (tid < a.given && token != -1)
            a.logprobs[(long long)r * a.given + tid] =
                known ? __fdiv_rn(given - m, a.T) - log_s : NAN;
        uint32_t bits = bad ? SV_DEV_BAD_ROW : 0;
        if (token != -1 && !known) bits |= SV_DEV_BAD_TOKEN;
        if (a.status && bits && (tid == 0 || token != -1)) atomicOr(a.status + r, bits);
        if (tid == 0 && a.normalizer)
            reinterpret_cast<float2*>(a.normalizer)[r] = make_float2(m, log_s);
        if (ENTROPY && tid == 0) a.entropy[r] = log_s - __fdiv_rn(t.u, t.s * a.T);
        const long long out = (long long)r * a.top;
        for (int i = (bad ? 0 : a.V) + tid; TOP && i < a.top; i += kThreads) {
            a.top_tokens[out + i] = -1;
            a.top_logprobs[out + i] = bad ? NAN : -INFINITY;
        }
        if (TOP && !bad) {
            // the lists side by side; an element's place is its place in its own list and how
            // many of each other one are above it
            const int all = G * a.top;
            for (int i = tid; i < all; i += kThreads)
                s_cand[i] = *cluster_at(&s_top[i % a.top], i / a.top);
            __syncthreads();
            for (int i = tid; i < all; i += kThreads) {
                const uint64_t k = s_cand[i];
                const int list = i / a.top;
                int above = i % a.top;
                for (int q = 0; q < G; ++q) {
                    if (q == list) continue;
                    int lo = 0, hi = a.top;  // how many of list q are above
                    while (lo < hi) {
                        const int mid = (lo + hi) / 2;
                        if (s_cand[q * a.top + mid] > k) lo = mid + 1;
                        else hi = mid;
                    }
                    above += lo;
                }
                if (!k || above >= a.top) continue;
                a.top_tokens[out + above] = place_of(k);
                a.top_logprobs[out + above] =
                    __fdiv_rn(from_ordered((uint32_t)(k >> 32)) - m, a.T) - log_s;
            }
        }
    }
    cluster_sync();  // nobody leaves while its share is being read
}

// ---------------------------------------------------------------- gradient

struct GradArgs {
    const void* logits;
    void* grad;
    long long stride, grad_stride;
    const int32_t* tokens;
    const float* normalizer;
    const float* entropy;
    const float* grad_logprobs;
    const float* grad_entropy;
    float T, c, c_low;  // c + c_low: log2(e) / T
    int V, given, parts;
    uint32_t* status;
};

constexpr int kGradBatches = 2;  // of kBatch vectors per thread: a CTA's part of a row

// Elements o .. o + kVec - 1 of two vectors side by side.
template <typename T> __device__ __forceinline__ uint4 shifted(const uint4& a, const uint4& b, int o) {
    constexpr int kPer = 4 / sizeof(T);  // elements per word
    uint32_t w[5];
    switch (o / kPer) {
        case 0: w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x; break;
        case 1: w[0] = a.y, w[1] = a.z, w[2] = a.w, w[3] = b.x, w[4] = b.y; break;
        case 2: w[0] = a.z, w[1] = a.w, w[2] = b.x, w[3] = b.y, w[4] = b.z; break;
        default: w[0] = a.w, w[1] = b.x, w[2] = b.y, w[3] = b.z, w[4] = b.w; break;
    }
    if (kPer == 2 && o % 2) {
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A part of a row per CTA: each logit read once, its gradient written once, in vectors of the
// gradient's row (where the logits lie at another place of a 16-byte word: two of theirs, shifted
// together: SHIFT).  With x = (l - m) / T in base 2 and less ln S, p = 2^x, a gradient is p (A + B x): A
// and B are the row's.  Then the places of given tokens again, with their own share (their logits
// are read before anything is written, so that the gradient may take the logits' place).
template <typename T, bool ENTROPY, bool SHIFT>
__global__ void __launch_bounds__(kThreads, 4) lp_grad_kernel(const GradArgs a) {
    using E = Elt<T>;
    constexpr int VW = E::kVec;
    __shared__ int s_token[kMaxGiven];
    __shared__ float s_g[kMaxGiven];
    const int tid = threadIdx.x, r = blockIdx.x / a.parts, part = blockIdx.x % a.parts;
    int token = -1;
    if (tid < a.given) token = a.tokens[(long long)r * a.given + tid];
    T* const out = (T*)a.grad + r * a.grad_stride;
    const Row<T> from((const T*)a.logits + r * a.stride, a.V), to(out, a.V);
    const int i0 = part * kThreads * kBatch * kGradBatches;
    const int i1 = min(to.vectors, i0 + kThreads * kBatch * kGradBatches);
    const bool live = __syncthreads_or(token != -1);
    uint4* const to16 = reinterpret_cast<uint4*>(out - to.skew);
    if (!live) {
        for (int i = i0 + tid; i < i1; i += kThreads) {
            if (to.whole(i)) {
                to16[i] = make_uint4(0, 0, 0, 0);
            } else {
                for (int e = 0; e < VW; ++e) {
                    const int v = i * VW + e - to.skew;
                    if (v >= 0 && v < a.V) out[v] = E::from(0.0f);
                }
            }
        }
        return;
    }
    const int off = SHIFT ? from.skew - to.skew : 0, by = off < 0 ? off + VW : off;  // shift of a vector
    const int back = off < 0 ? 1 : 0;
    // Vectors that lie wholly in the row, as what they are made of does; the others, two at each
    // end at most, go element by element.
    auto fast = [&](int i) {
        return to.whole(i) &&
               (off == 0 || (from.whole(i - back) && i - back >= 0 && from.whole(i - back + 1)));
    };
    auto load = [&](int i) -> uint4 {
        if (i >= i1 || !fast(i)) return make_uint4(0, 0, 0, 0);
        if (off == 0) return ld_own16(from.at(i));
        return shifted<T>(ld_own16(from.at(i - back)), ld_own16(from.at(i - back + 1)), by);
    };
    uint4 x[kBatch];
#pragma unroll
    for (int q = 0; q < kBatch; ++q) x[q] = load(i0 + tid + q * kThreads);

    const float2 z = reinterpret_cast<const float2*>(a.normalizer)[r];
    const float m = z.x, log_s = z.y;
    float H = 0.0f, gh = 0.0f;
    if (ENTROPY) H = a.entropy[r], gh = a.grad_entropy[r];
    bool bad = !(fabsf(m) < INFINITY && fabsf(log_s) < INFINITY);
    if (tid < a.given) {
        s_token[tid] = token;
        s_g[tid] = token != -1 ? a.grad_logprobs[(long long)r * a.given + tid] : 0.0f;
    }
    // (of given tokens: this thread's place is in this part)
    const int at = token < 0 || token >= a.V ? -1 : (token + to.skew) / VW;
    bool mine = at >= i0 && at < i1;
    const float own = mine ? E::get(from.row + token) : 0.0f;
    const bool bad_token = __syncthreads_or(token < -1 || token >= a.V);
    if (part == 0 && tid == 0 && a.status && (bad || bad_token))
        atomicOr(a.status + r, (bad ? SV_DEV_BAD_ROW : 0) | (bad_token ? SV_DEV_BAD_TOKEN : 0));
    bad |= bad_token;
    float sum = 0.0f;
    for (int k = 0; k < a.given; ++k) sum += s_g[k];
    const float base = log_s * 1.4426950408889634f;
    const float A = bad ? NAN : -__fdiv_rn(ENTROPY ? fmaf(gh, H, sum) : sum, a.T);
    const float B = ENTROPY ? -__fdiv_rn(gh * 0.6931471805599453f, a.T) : 0.0f;
    auto grad = [&](float l) -> float {
        const float d = l - m;
        // (the low half of the factor where the gradient has the bits to show it)
        const float y = fmaf(d, a.c, sizeof(T) == 4 ? fmaf(d, a.c_low, -base) : -base);
        const float p = ex2(y);
        return p * (ENTROPY ? fmaf(B, max_nan(y, -1e4f), A) : A);
    };
    for (int n = 0;; ++n) {
        const int i = i0 + n * kThreads * kBatch + tid;
        uint4 next[kBatch];
        if (n + 1 < kGradBatches) {
#pragma unroll
            for (int q = 0; q < kBatch; ++q) next[q] = load(i + (kBatch + q) * kThreads);
        }
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            const int k = i + q * kThreads;
            if (k >= i1 || !fast(k)) continue;
            float f[VW];
            E::unpack(x[q], f);
#pragma unroll
            for (int e = 0; e < VW; ++e) f[e] = grad(f[e]);
            to16[k] = E::pack(f);
        }
        if (n + 1 == kGradBatches) break;
#pragma unroll
        for (int q = 0; q < kBatch; ++q) x[q] = next[q];
    }
    if (tid < 4 * VW) {
        const int n = tid / VW, i = n < 2 ? n : to.vectors - 4 + n;
        const int v = i * VW + tid % VW - to.skew;
        if (i >= i0 && i < i1 && (n < 2 || i > 1) && !fast(i) && v >= 0 && v < a.V)
            out[v] = E::from(grad(E::get(from.row + v)));
    }
    __syncthreads();
    if (mine && !bad) {
        float g = 0.0f;
        for (int k = 0; k < a.given; ++k) {
            if (s_token[k] != token) continue;
            if (k < tid) mine = false;  // an equal one before it writes
            g += s_g[k];
        }
        if (mine) out[token] = E::from(grad(own) + __fdiv_rn(g, a.T));
    }
}

// ---------------------------------------------------------------- host

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

static sv_status device_ok(int* sms) {
    static std::mutex mu;
    static int known[64];  // 0 unknown, -1 another device
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SV_ERR_CUDA;
    if (dev < 0 || dev >= 64) return SV_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lk(mu);
    if (!known[dev]) {
        int major = 0, minor = 0, n = -1;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
            return SV_ERR_CUDA;
        if (major == 10 && minor == 3 &&
            cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return SV_ERR_CUDA;
        known[dev] = n;
    }
    if (known[dev] < 0) return SV_ERR_UNSUPPORTED;
    *sms = known[dev];
    return SV_OK;
}

static sv_status check_rows(const void* logits, sv_dtype dtype, int64_t stride,
                            const int32_t* tokens, float T, int rows, int V, int given) {
    if (dtype != SV_BF16 && dtype != SV_F32) return SV_ERR_INVALID_ARG;
    if (rows < 0 || V < 1 || given < 1 || stride < V) return SV_ERR_INVALID_ARG;
    if (!(T > 0.0f) || !std::isfinite(T)) return SV_ERR_INVALID_ARG;
    if (V > kMaxV || given > kMaxGiven || rows >= (1 << 27) || stride >= (1ll << 40) ||
        (long double)rows * stride >= (long double)(1ll << 40))
        return SV_ERR_UNSUPPORTED;
    if (rows > 0 && (!logits || !tokens)) return SV_ERR_INVALID_ARG;
    if (!aligned16(logits) || !aligned16(tokens)) return SV_ERR_INVALID_ARG;
    return SV_OK;
}

// log2(e) / T as a sum of two floats, the second positive, so that it may be multiplied with
// -infinity too; for the smallest T the largest float (0 times infinity is NaN).
static void base2(float T, float* high, float* low) {
    const double c = std::fmin(1.4426950408889634 / T, (double)FLT_MAX);
    *high = (float)c;
    while (!((double)*high < c)) *high = std::nextafterf(*high, 0.0f);
    *low = std::fmax((float)(c - *high), std::nextafterf(0.0f, 1.0f));
}

template <typename K, typename A>
static sv_status launch(K kernel, long long ctas, int cluster, cudaStream_t stream, const A& a) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace svlp

using namespace svlp;

extern "C" {

size_t spec_logprobs_workspace_size(int rows, int V, sv_dtype dtype, int given, int top) {
    if (rows < 0 || rows >= (1 << 27) || V < 1 || V > kMaxV || given < 1 || given > kMaxGiven ||
        top < 0 || top > kMaxTop || (dtype != SV_BF16 && dtype != SV_F32))
        return 0;
    return 256;
}

sv_status spec_logprobs(const void* logits, sv_dtype dtype, int64_t row_stride,
                        const int32_t* tokens, float T, int rows, int V, int given, int top,
                        float* logprobs, float* normalizer, float* entropy, int32_t* top_tokens,
                        float* top_logprobs, void* ws, size_t ws_bytes, uint32_t* status,
                        cudaStream_t stream) {
    sv_status st = check_rows(logits, dtype, row_stride, tokens, T, rows, V, given);
    if (st != SV_OK) return st;
    if (top < 0) return SV_ERR_INVALID_ARG;
    if (top > kMaxTop) return SV_ERR_UNSUPPORTED;
    if (rows > 0 && (!logprobs || (top && (!top_tokens || !top_logprobs))))
        return SV_ERR_INVALID_ARG;
    for (const void* p : {(const void*)logprobs, (const void*)normalizer, (const void*)entropy,
                          (const void*)top_tokens, (const void*)top_logprobs, (const void*)status,
                          (const void*)ws})
        if (!aligned16(p)) return SV_ERR_INVALID_ARG;
    if (!ws || ws_bytes < spec_logprobs_workspace_size(rows, V, dtype, given, top))
        return SV_ERR_WORKSPACE;
    if (rows == 0) return SV_OK;
    int sms;
    if ((st = device_ok(&sms)) != SV_OK) return st;
    Args a = {logits, row_stride, tokens, T, 0.0f, 0.0f, V, given, top, logprobs, normalizer,
              entropy, top_tokens, top_logprobs, status};
    base2(T, &a.c, &a.c_low);
    int G = 1;
    while (G < kMaxCluster && (long long)rows * G < 4 * sms && V / G >= 16384) G *= 2;
    const long long ctas = (long long)rows * G;
    auto typed = [&](auto t) {
        using E = decltype(t);
        if (entropy)
            return top ? launch(lp_kernel<E, true, true>, ctas, G, stream, a)
                       : launch(lp_kernel<E, true, false>, ctas, G, stream, a);
        return top ? launch(lp_kernel<E, false, true>, ctas, G, stream, a)
                   : launch(lp_kernel<E, false, false>, ctas, G, stream, a);
    };
    return dtype == SV_BF16 ? typed(__nv_bfloat16()) : typed(0.0f);
}

sv_status spec_logprobs_grad(const void* logits, sv_dtype dtype, int64_t row_stride,
                             const int32_t* tokens, const float* normalizer, const float* entropy,
                             const float* grad_logprobs, const float* grad_entropy, float T,
                             int rows, int V, int given, void* grad_logits, int64_t grad_stride,
                             uint32_t* status, cudaStream_t stream) {
    sv_status st = check_rows(logits, dtype, row_stride, tokens, T, rows, V, given);
    if (st != SV_OK) return st;
    if (grad_stride < V) return SV_ERR_INVALID_ARG;
    if (grad_stride >= (1ll << 40) || (long double)rows * grad_stride >= (long double)(1ll << 40))
        return SV_ERR_UNSUPPORTED;
    if (rows > 0 && (!normalizer || !grad_logprobs || !grad_logits || (grad_entropy && !entropy)))
        return SV_ERR_INVALID_ARG;
    for (const void* p : {(const void*)normalizer, (const void*)entropy, (const void*)grad_logprobs,
                          (const void*)grad_entropy, (const void*)grad_logits, (const void*)status})
        if (!aligned16(p)) return SV_ERR_INVALID_ARG;
    if (logits && logits == grad_logits && rows > 1 && row_stride != grad_stride)
        return SV_ERR_INVALID_ARG;
    if (rows == 0) return SV_OK;
    int sms;
    if ((st = device_ok(&sms)) != SV_OK) return st;
    // (of vectors; a row may begin inside of one)
    const int width = dtype == SV_BF16 ? 8 : 4, part = kThreads * kBatch * kGradBatches;
    GradArgs a = {logits, grad_logits, row_stride, grad_stride, tokens, normalizer, entropy,
                  grad_logprobs, grad_entropy, T, 0.0f, 0.0f, V, given,
                  ((V + width - 1 + width - 1) / width + part - 1) / part, status};
    base2(T, &a.c, &a.c_low);
    const long long ctas = (long long)rows * a.parts;
    if (ctas >= (1ll << 31)) return SV_ERR_UNSUPPORTED;
    const bool shift = rows > 1 && (row_stride - grad_stride) % width != 0;
    auto typed = [&](auto t) {
        using E = decltype(t);
        if (grad_entropy)
            return shift ? launch(lp_grad_kernel<E, true, true>, ctas, 1, stream, a)
                         : launch(lp_grad_kernel<E, true, false>, ctas, 1, stream, a);
        return shift ? launch(lp_grad_kernel<E, false, true>, ctas, 1, stream, a)
                     : launch(lp_grad_kernel<E, false, false>, ctas, 1, stream, a);
    };
    return dtype == SV_BF16 ? typed(__nv_bfloat16()) : typed(0.0f);
}

}  // extern "C"
