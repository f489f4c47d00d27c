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

constexpr int kThreads = 256;    // of the gradient's CTAs
constexpr int kBatch = 4;        // 16-byte vectors of a thread in flight there
constexpr int kMaxV = 1 << 21;
constexpr int kMaxGiven = SV_LOGPROBS_MAX_GIVEN;
constexpr int kMaxTop = SV_LOGPROBS_MAX_TOP;
constexpr int kGroups = 128;     // of threads, whose largest elements make the alternatives' bound
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
// A 64-bit word of shared memory, and two of them from a 16-byte boundary.
__device__ __forceinline__ uint64_t lds64(uint32_t at) {
    uint64_t x;
    asm volatile("ld.shared.u64 %0, [%1];" : "=l"(x) : "r"(at) : "memory");
    return x;
}
__device__ __forceinline__ void lds64x2(uint64_t* x, uint32_t at) {
    asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(x[0]), "=l"(x[1]) : "r"(at) : "memory");
}
__device__ __forceinline__ void sts64(uint32_t at, uint64_t x) {
    asm volatile("st.shared.u64 [%0], %1;" ::"r"(at), "l"(x) : "memory");
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
__device__ __forceinline__ void add(Stats& a, const Stats& b, float c, float c_low) {
    const float m = fmaxf(a.m, b.m);
    const float da = a.m == m || a.m == -INFINITY ? 0.0f : a.m - m;
    const float db = b.m == m || b.m == -INFINITY ? 0.0f : b.m - m;
    // (the small product first, so that the exponent is rounded once; a side's factor is all of its
    // sum's, so that the low half tells here too)
    const float fa = ex2(fmaf(da, c, da * c_low)), fb = ex2(fmaf(db, c, db * c_low));
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
// maximum and sums of a softmax; joined through distributed shared memory.  A thread's vectors come
// through a ring of its own in shared memory (asynchronous 16-byte copies), so that many are on
// their way whatever the registers hold, and the CTAs of an SM hide each other's beginnings and
// ends.
//
// Alternatives.  Each thread knows its largest element, the first batch of vectors that it is in
// and the largest element of its others.  Of the largest elements of 128 groups of threads the
// top-th is a bound: as many elements are at or above it, and these are in the batches of the
// threads whose own maximum reaches it, about as many again.  Those threads look into their batch
// again, and where another of theirs may reach the bound too (equal ones: by its place, which is
// behind the first), their warp goes through all of them.  The elements that reach the bound are
// put in order by counting, 256 at most: of more, those below the top-th of the first 256 go first.
// Rank 0 joins the lists of the cluster's CTAs.
//
// Measured: 4096 rows of 128256 in bf16 without entropy and alternatives 156 us, 6.7 TB/s (memory);
// 300 of 65537 in fp32 with eight alternatives 18.6 us, 576 of 151936 with 20 41 us (38.5 where
// half of them are without tokens), nine of 256000 with five 11.4 us (the steps behind the row wait
// for one another: 3 us, 7 where others keep the SM busy).  Choices, measured before the kernel
// was launched ahead of the end of the one before it: 157 us on the first of these, 167 with the
// entropy, 205 with it and 20 alternatives (instructions: the second product per element, and a
// warp's turn of many small steps at the end of each row).  Stages of two vectors instead of four,
// five CTAs per SM: 162, 178 and 220 us; 128 threads: 160, 164 and 211 us, but 32 instead of 24 us
// for nine rows of 256000 with five alternatives by one CTA each.
constexpr int kLpThreads = 256, kLpWarps = kLpThreads / 32;
constexpr int kLpBatch = 4;      // vectors of a thread per stage
constexpr int kLpStages = 3;
constexpr int kLpResident = 4;   // CTAs per SM
constexpr int kLpRing = kLpStages * kLpBatch * kLpThreads * 16;  // bytes

template <typename T, bool ENTROPY, bool TOP>
__global__ void __launch_bounds__(kLpThreads, kLpResident) lp_kernel(const Args a) {
    using E = Elt<T>;
    constexpr int VW = E::kVec, B = kLpBatch, S = kLpStages;
    extern __shared__ __align__(16) uint64_t s_mem[];  // the ring; then candidates
    __shared__ __align__(16) uint64_t s_group[kGroups];
    __shared__ uint64_t s_top[kMaxTop], s_bound;
    __shared__ Stats s_warp[kLpWarps], s_stats;
    __shared__ int s_count;
    static_assert(kLpRing / S >= kCandidates * 8 && S > 1, "candidates in the ring's first stage");
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int G = cluster_size(), rank = cluster_rank();
    const int r = blockIdx.x / G;

    // (launched while the kernel before ends; nothing is read before it has)
    cudaGridDependencySynchronize();
    cudaTriggerProgrammaticLaunchCompletion();
    int token = -1;
    if (tid < a.given) token = a.tokens[(long long)r * a.given + tid];
    if (!__syncthreads_or(token != -1)) return;  // (the whole cluster)
    const Row<T> row((const T*)a.logits + r * a.stride, a.V);
    // whole vectors here; the two that the row may share with others by a thread each
    const int w0 = row.skew != 0, w1 = (a.V + row.skew) / VW, whole = max(w1 - w0, 0);
    const int i0 = w0 + (int)((long long)whole * rank / G);
    const int i1 = w0 + (int)((long long)whole * (rank + 1) / G);
    const uint32_t cand = (uint32_t)__cvta_generic_to_shared(s_mem), ring = cand + tid * 16;
    const uint32_t group = (uint32_t)__cvta_generic_to_shared(s_group);
    // B of this thread's vectors, from k on, into a stage of the ring; vector q of a stage.
    auto copy = [&](int k, int slot) {
#pragma unroll
        for (int q = 0; q < B; ++q, k += kLpThreads) {
            if (k < i1)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                    ring + (slot * B + q) * kLpThreads * 16), "l"(row.at(k)) : "memory");
        }
    };
    auto copied = [&](int slot, int q) {
        uint4 v;
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "r"(ring + (slot * B + q) * kLpThreads * 16) : "memory");
        return v;
    };
    auto issue = [&](int n, int slot) {
        copy(i0 + tid + n * B * kLpThreads, slot);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int n = 0; n < S - 1; ++n) issue(n, n);
    const bool known = token >= 0 && token < a.V;
    const float given = rank == 0 && known ? E::get(row.row + token) : 0.0f;

    // The warp's reference and this thread's sums; its largest element, the batch of vectors that
    // holds it first, and the largest element of its other batches.
    Stats st = {-INFINITY, 0.0f, 0.0f};
    float mine = -INFINITY, next = -INFINITY;
    int best = 0;
    auto take = [&](const uint4 (&v)[B], int n) {
        float most = E::largest(v[0]);
#pragma unroll
        for (int q = 1; q < B; ++q) most = fmaxf(most, E::largest(v[q]));
        if (TOP) {
            best = most > mine ? n : best;
            next = fmaxf(next, fminf(most, mine));
            mine = fmaxf(mine, most);
        }
        if (__any_sync(~0u, most > st.m)) {  // all lanes follow the largest of theirs
#pragma unroll
            for (int k = 16; k; k >>= 1) most = fmaxf(most, __shfl_xor_sync(~0u, most, k));
            add(st, Stats{most, 0.0f, 0.0f}, a.c, a.c_low);
        }
        const float2 less = both(st.m == -INFINITY ? 0.0f : -st.m);
        float2 s = make_float2(0.0f, 0.0f), u = s;
#pragma unroll
        for (int q = 0; q < B; ++q) {
            float x[VW];
            E::unpack(v[q], x);
#pragma unroll
            for (int e = 0; e < VW; e += 2) {
                float2 d = add2(make_float2(x[e], x[e + 1]), less);
                float2 p = fma2(d, both(a.c), mul2(d, both(a.c_low)));  // rounded once
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
    };
    const uint4 none = make_uint4(E::kLowest, E::kLowest, E::kLowest, E::kLowest);
    const int stages = (i1 - i0 + B * kLpThreads - 1) / (B * kLpThreads);
    // (the shared vectors: the first thread's batch before its others, the last one's behind)
    const bool head = rank == 0 && w0 == 1;
    const bool tail = rank == G - 1 && row.vectors > max(w0, w1);
    if (head && w == 0) {
        uint4 v[B];
#pragma unroll
        for (int q = 0; q < B; ++q) v[q] = none;
        if (tid == 0) v[0] = row.load(0);
        take(v, -1);
    }
    int slot = 0;
    for (int n = 0; n < stages; ++n) {
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
        uint4 v[B];
#pragma unroll
        for (int q = 0; q < B; ++q) {
            v[q] = none;
            if (i0 + tid + (n * B + q) * kLpThreads < i1) v[q] = copied(slot, q);
        }
        // (into the place of the stage before this one)
        issue(n + S - 1, slot == 0 ? S - 1 : slot - 1);
        slot = slot == S - 1 ? 0 : slot + 1;
        take(v, n);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (tail && w == kLpWarps - 1) {
        uint4 v[B];
#pragma unroll
        for (int q = 0; q < B; ++q) v[q] = none;
        if (tid == kLpThreads - 1) v[0] = row.load(row.vectors - 1);
        take(v, stages);
    }
#pragma unroll
    for (int k = 16; k; k >>= 1) {
        st.s += __shfl_xor_sync(~0u, st.s, k);
        if (ENTROPY) st.u += __shfl_xor_sync(~0u, st.u, k);
    }
    if (lane == 0) s_warp[w] = st;
    // The first and the last vector of batch n of thread t.
    auto first_of = [&](int t, int n) {
        return n < 0 ? 0 : n == stages ? row.vectors - 1 : i0 + t + n * B * kLpThreads;
    };
    bool some = false;  // whether this thread has had elements of the row
    int lead = 0;       // its first batch
    // Threads per group: few groups are quicker to put in order, and bring few elements more than
    // are wanted (24 of 64 groups: about 30).
    const int share = a.top <= 24 ? 2 * kLpThreads / kGroups : kLpThreads / kGroups;
    if (TOP) {
        some = i0 + tid < i1 || (head && tid == 0) || (tail && tid == kLpThreads - 1);
        lead = head && tid == 0 ? -1 : i0 + tid < i1 ? 0 : stages;
        if (mine == -INFINITY) best = lead;
        // As many elements as there are groups are at or above their largest elements' keys, of
        // which the last place of the batch is known only.
        const int end = first_of(tid, best) + (best < 0 || best == stages ? 0 : B - 1) * kLpThreads;
        uint64_t largest = some ? key_of(mine, min(min(end, row.vectors) * VW + VW - 1 - row.skew,
                                                   a.V - 1)) : 0;
        for (int k = 1; k < share; k *= 2) {
            const uint64_t o = __shfl_xor_sync(~0u, largest, k);
            largest = o > largest ? o : largest;
        }
        if (tid % share == 0) s_group[tid / share] = largest;
        if (tid < kMaxTop) s_top[tid] = 0;
        if (tid == 0) s_bound = 0, s_count = 0;
    }
    __syncthreads();
    if (w == kLpWarps - 1) {
        Stats t = s_warp[lane % kLpWarps];
#pragma unroll
        for (int k = kLpWarps / 2; k; k >>= 1) {
            Stats o;
            o.m = __shfl_xor_sync(~0u, t.m, k);
            o.s = __shfl_xor_sync(~0u, t.s, k);
            o.u = __shfl_xor_sync(~0u, t.u, k);
            add(t, o, a.c, a.c_low);
        }
        if (lane == 0) s_stats = t;
    }
    if (TOP) {
        // a group's place among all: counted by its threads, a share of the groups each
        const int part = kLpThreads / share / share / 2;
        const uint64_t p = lds64(group + tid / share * 8);
        int places = 0;  // how many are above, and (from bit 16 on) how many are not below
#pragma unroll 8
        for (int k = 0; k < part; ++k) {
            uint64_t o[2];
            lds64x2(o, group + (tid % share * part + k) * 16);
#pragma unroll
            for (int e = 0; e < 2; ++e) places += (o[e] > p ? 1 : 0) + (o[e] >= p ? 1 << 16 : 0);
        }
        for (int k = 1; k < share; k *= 2) places += __shfl_xor_sync(~0u, places, k);
        // (equal keys: of threads whose batches end with the row)
        if (p && (places & 0xffff) < a.top && places >> 16 >= a.top) s_bound = p;
        // What nothing has to be looked for below; the elements that reach it; where they are more
        // than there is room for (many that are equal, or large ones that lie together), the top-th
        // of those that found room is the next, higher bound.
        auto from = [&](float x, int n) {  // the highest key that an element of batch n may have
            return key_of(x, max(first_of(tid, n) * VW - row.skew, 0));
        };
        const uint64_t highest = some ? from(mine, best) : 0;
        // of the other batches: one that has the largest element too comes behind the first
        const uint64_t other = from(next, next == mine || best == lead ? best + 1 : lead);
        for (;;) {
            __syncthreads();
            const uint64_t bound = s_bound;
            auto look = [&](float x, int at) {
                const uint64_t k = key_of(x, at);
                if (k < bound) return;
                const int n = atomicAdd(&s_count, 1);
                if (n < kCandidates) sts64(cand + n * 8, k);
            };
            const bool reaches = some && highest >= bound;
            const bool more = reaches && other >= bound;
            // Those threads' batches: up to eight of a warp's one after the other, a lane per
            // element; more of them at once, each thread its own (a row of equal logits, where all
            // 32 are looked into twice: 18 us instead of 74; rows like a model's have one to three,
            // which the first way takes half a microsecond each for and the second 1.6 together).
            uint32_t few = __ballot_sync(~0u, reaches && !more);
            if (__popc(few) <= 8) {
#pragma unroll 1
                for (; few; few &= few - 1) {
                    const int t = __ffs(few) - 1, n = __shfl_sync(~0u, best, t);
                    const bool one = n < 0 || n == stages;
#pragma unroll
                    for (int e = lane; e < B * VW; e += 32) {
                        const int i = first_of(w * 32 + t, n) + e / VW * kLpThreads;
                        const int at = i * VW + e % VW - row.skew;
                        if (at >= 0 && at < a.V && (one ? e < VW : i < i1))
                            look(E::get(row.row + at), at);
                    }
                }
            } else if (reaches && !more) {
                const bool one = best < 0 || best == stages;
                const int i = first_of(tid, best), end = one ? i + 1 : i1;
                if (!one) copy(i, 1);  // (behind the candidates)
                asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 1
                for (int q = 0; q < B && i + q * kLpThreads < end; ++q) {
                    float x[VW];
                    E::unpack(one ? row.load(i) : copied(1, q), x);
#pragma unroll
                    for (int e = 0; e < VW; ++e) {
                        const int at = (i + q * kLpThreads) * VW + e - row.skew;
                        if (!one || (at >= 0 && at < a.V)) look(x[e], at);
                    }
                }
            }
            // and of those threads' vectors that have more than one
#pragma unroll 1
            for (uint32_t all = __ballot_sync(~0u, more); all; all &= all - 1) {
                const int t = w * 32 + __ffs(all) - 1;
                const int edge = head && t == 0                ? 0
                                 : tail && t == kLpThreads - 1 ? row.vectors - 1
                                                               : -1;
                if (edge >= 0 && lane < VW) {
                    const int at = edge * VW + lane - row.skew;
                    if (at >= 0 && at < a.V) look(E::get(row.row + at), at);
                }
#pragma unroll 1
                for (int i = i0 + t + lane * kLpThreads; i < i1; i += 32 * kLpThreads) {
                    float x[VW];
                    E::unpack(ld_stream16(row.at(i)), x);
#pragma unroll
                    for (int e = 0; e < VW; ++e) look(x[e], i * VW + e - row.skew);
                }
            }
            __syncthreads();
            const int n = s_count;
            for (int here = min(n, kCandidates);;) {
                // The places of the candidates, or of the first 256, counted by eight threads for
                // each; none below the top-th of these is wanted.
                const int some = min(here, kLpThreads), sub = tid % 8;
                for (int i0 = 0; i0 < some; i0 += kLpThreads / 8) {
                    const int i = i0 + tid / 8;
                    const uint64_t k = i < some ? lds64(cand + i * 8) : 0;
                    int before = 0;
#pragma unroll 4
                    for (int j = sub; j < some; j += 8) before += lds64(cand + j * 8) > k;
#pragma unroll
                    for (int x = 1; x < 8; x *= 2) before += __shfl_xor_sync(~0u, before, x);
                    if (sub || i >= some || before >= a.top) continue;
                    s_top[before] = k;
                    if (before == a.top - 1) s_bound = k;
                }
                if (here == some) break;
                uint64_t k[kCandidates / kLpThreads];
#pragma unroll
                for (int q = 0; q < kCandidates / kLpThreads; ++q) {
                    const int i = tid + q * kLpThreads;
                    k[q] = i < here ? lds64(cand + i * 8) : 0;
                }
                __syncthreads();
                const uint64_t least = s_bound;
                if (tid == 0) s_count = 0;
                __syncthreads();
#pragma unroll
                for (int q = 0; q < kCandidates / kLpThreads; ++q)
                    if (k[q] >= least) sts64(cand + atomicAdd(&s_count, 1) * 8, k[q]);
                __syncthreads();
                here = s_count;
            }
            if (n <= kCandidates) break;
            __syncthreads();
            if (tid == 0) s_count = 0;
        }
    }
    if (G > 1) cluster_sync();
    else __syncthreads();
    if (rank == 0) {
        Stats t = s_stats;
        for (int k = 1; k < G; ++k) add(t, *cluster_at(&s_stats, k), a.c, a.c_low);
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
        for (int i = (bad ? 0 : a.V) + tid; TOP && i < a.top; i += kLpThreads) {
            a.top_tokens[out + i] = -1;
            a.top_logprobs[out + i] = bad ? NAN : -INFINITY;
        }
        if (TOP && !bad) {
            auto tell = [&](int place, uint64_t k) {
                a.top_tokens[out + place] = place_of(k);
                a.top_logprobs[out + place] =
                    __fdiv_rn(from_ordered((uint32_t)(k >> 32)) - m, a.T) - log_s;
            };
            if (G == 1) {
                if (tid < min(a.top, a.V)) tell(tid, s_top[tid]);
            } else {
                // the lists side by side; an element's place is its place in its own list and how
                // many of each other one are above it
                const int all = G * a.top;
                for (int i = tid; i < all; i += kLpThreads)
                    sts64(cand + i * 8, *cluster_at(&s_top[i % a.top], i / a.top));
                __syncthreads();
                for (int i = tid; i < all; i += kLpThreads) {
                    const uint64_t k = lds64(cand + i * 8);
                    const int list = i / a.top;
                    int before = i % a.top;
                    for (int q = 0; q < G; ++q) {
                        if (q == list) continue;
                        int lo = 0, hi = a.top;  // how many of list q are above
                        while (lo < hi) {
                            const int mid = (lo + hi) / 2;
                            if (lds64(cand + (q * a.top + mid) * 8) > k) lo = mid + 1;
                            else hi = mid;
                        }
                        before += lo;
                    }
                    if (k && before < a.top) tell(before, k);
                }
            }
        }
    }
    if (G > 1) cluster_sync();  // nobody leaves while its share is being read
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
template <typename T>
__device__ __forceinline__ uint4 shifted(const uint4& a, const uint4& b, int o) {
    constexpr int kPer = 4 / sizeof(T);  // elements per word
    const bool two = o / kPer & 2, one = o / kPer & 1;
    uint32_t w[6] = {two ? a.z : a.x, two ? a.w : a.y, two ? b.x : a.z,
                     two ? b.y : a.w, two ? b.z : b.x, two ? b.w : b.y};
#pragma unroll
    for (int k = 0; k < 5; ++k) w[k] = one ? w[k + 1] : w[k];
    if (kPer == 2) {
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], o % 2 * 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A part of a row per CTA: each logit read once, its gradient written once, in vectors of the
// gradient's row (where the logits lie at another place of a 16-byte word: two of theirs, shifted
// together: SHIFT).  With x = (l - m) / T in base 2 and less ln S, p = 2^x, a gradient is
// p (A + B x): A and B are the row's.  Then the places of given tokens again, with their own share
// (their logits are read before anything is written, so that the gradient may take the logits'
// place).
//
// Bound by memory: 4096 rows of 128256 in bf16 310 us, 6.8 TB/s (all of them read); 1024 of 65537
// in fp32 with the entropy and 32 tokens each 87 us, 6.2 TB/s.  Shifted, the first takes 352 us,
// and in fp32 630 where rows that lie alike take 598: a warp's vectors lie side by side and a lane
// has what lies behind its own from its neighbour (two loads per vector, each waited for by its
// shift: 528 and 1095 us; from the neighbour, but with the next batch under way and thus three
// CTAs per SM: 426 and 814; four CTAs without it 357 and 647, five 352 and 630).
template <typename T, bool ENTROPY, bool SHIFT>
__global__ void __launch_bounds__(kThreads, SHIFT ? 5 : 4) lp_grad_kernel(const GradArgs a) {
    using E = Elt<T>;
    constexpr int VW = E::kVec;
    __shared__ int s_token[kMaxGiven];
    __shared__ float s_g[kMaxGiven];
    const int tid = threadIdx.x, r = blockIdx.x / a.parts, part = blockIdx.x % a.parts;
    cudaGridDependencySynchronize();
    cudaTriggerProgrammaticLaunchCompletion();
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
    // how much further into a vector the logits' elements lie, and in which of two vectors
    const int off = SHIFT ? from.skew - to.skew : 0, by = off < 0 ? off + VW : off;
    const int back = off < 0 ? 1 : 0;
    // Vectors that lie wholly in the row, as what they are made of does; the others, two at each
    // end at most, go element by element.
    auto fast = [&](int i) {
        return to.whole(i) &&
               (off == 0 || (from.whole(i - back) && i - back >= 0 && from.whole(i - back + 1)));
    };
    // Vector q of this thread in batch n.  Shifted ones are a warp's side by side: what lies behind
    // a lane's is its neighbour's, and the warp's last has one vector more.
    const int lane = tid % 32;
    auto place = [&](int n, int q) {
        return i0 + n * kThreads * kBatch +
               (SHIFT ? (tid - lane) * kBatch + q * 32 + lane : q * kThreads + tid);
    };
    auto load = [&](int i) {
        if (!SHIFT) return i < i1 && fast(i) ? ld_own16(from.at(i)) : uint4();
        const int j = i - back;  // (i may lie one behind this CTA's part)
        return i <= i1 && j >= 0 && from.whole(j) ? ld_stream16(from.at(j)) : uint4();
    };
    auto behind = [&](int n) { return lane == 31 ? load(place(n, kBatch - 1) + 1) : uint4(); };
    uint4 x[kBatch], last = {};
#pragma unroll
    for (int q = 0; q < kBatch; ++q) x[q] = load(place(0, q));
    if (SHIFT) last = behind(0);

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
        uint4 next[kBatch];
        if (!SHIFT && n + 1 < kGradBatches) {
#pragma unroll
            for (int q = 0; q < kBatch; ++q) next[q] = load(place(n + 1, q));
        }
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            const int k = place(n, q);
            uint4 v = x[q];
            if (SHIFT) {
                const uint4 y = lane ? v : q + 1 < kBatch ? x[(q + 1) % kBatch] : last;
                const int up = (lane + 1) % 32;
                uint4 o = {__shfl_sync(~0u, y.x, up), __shfl_sync(~0u, y.y, up),
                           __shfl_sync(~0u, y.z, up), __shfl_sync(~0u, y.w, up)};
                if (q + 1 == kBatch && lane == 31) o = last;
                v = shifted<T>(v, o, by);
            }
            if (k >= i1 || !fast(k)) continue;
            float f[VW];
            E::unpack(v, f);
#pragma unroll
            for (int e = 0; e < VW; ++e) f[e] = grad(f[e]);
            to16[k] = E::pack(f);
        }
        if (n + 1 == kGradBatches) break;
#pragma unroll
        for (int q = 0; q < kBatch; ++q) x[q] = SHIFT ? load(place(n + 1, q)) : next[q];
        if (SHIFT) last = behind(n + 1);
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

// The ring of lp_kernel is more than a kernel gets unasked.
template <typename T> static bool lp_setup() {
    bool ok = true;
    for (auto k : {lp_kernel<T, false, false>, lp_kernel<T, false, true>, lp_kernel<T, true, false>,
                   lp_kernel<T, true, true>})
        ok = ok && cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kLpRing) ==
                       cudaSuccess;
    return ok;
}

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
        if (n > 0 && !(lp_setup<__nv_bfloat16>() && lp_setup<float>())) return SV_ERR_CUDA;
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
    // (so that 1 / T, T times a sum and a far element's share of one stay within fp32)
    if (T < 0x1p-100f || T > 0x1p100f) return SV_ERR_UNSUPPORTED;
    if (V > kMaxV || given > kMaxGiven || rows >= (1 << 27) || stride >= (1ll << 40) ||
        (long double)rows * stride >= (long double)(1ll << 40))
        return SV_ERR_UNSUPPORTED;
    if (rows > 0 && (!logits || !tokens)) return SV_ERR_INVALID_ARG;
    if (!aligned16(logits) || !aligned16(tokens)) return SV_ERR_INVALID_ARG;
    return SV_OK;
}

// log2(e) / T as a sum of two floats, the second positive, so that it may be multiplied with
// -infinity too (0 times infinity is NaN).
static void base2(float T, float* high, float* low) {
    const double c = 1.4426950408889634 / T;
    *high = (float)c;
    while (!((double)*high < c)) *high = std::nextafterf(*high, 0.0f);
    *low = std::fmax((float)(c - *high), std::nextafterf(0.0f, 1.0f));
}

template <typename K, typename A>
static sv_status launch(K kernel, int threads, int smem, long long ctas, int cluster,
                        cudaStream_t stream, const A& a) {
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = cluster;
    attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attrs;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
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
    // A cluster per row while its CTAs have SMs of their own and runs worth a CTA's beginning and
    // end (9 rows of 256000, 5 alternatives: G = 1 20.4 us, 2 16.5, 4 14.5, 8 14.2; 40 of 128256:
    // 16.6, 16.0, 16.6, 18.5; 5 of 32000: 8.5, 10.4).  More rows: a CTA each.  (300 of 65536, all
    // with tokens: 14.3 us, two each 18.4; 576: 23 and 35; 576 of 151936: 41 and 52.  Where half of
    // them hold none, those that do meet on some SMs by chance, and two each take 30 instead of 39
    // there, but which rows hold tokens is known on the device only.)
    int G = 1;
    while (G < kMaxCluster && 2ll * rows * G <= sms && V / G >= 49152) G *= 2;
    const long long ctas = (long long)rows * G;
    auto typed = [&](auto t) {
        using E = decltype(t);
        if (entropy)
            return top ? launch(lp_kernel<E, true, true>, kLpThreads, kLpRing, ctas, G, stream, a)
                       : launch(lp_kernel<E, true, false>, kLpThreads, kLpRing, ctas, G, stream, a);
        return top ? launch(lp_kernel<E, false, true>, kLpThreads, kLpRing, ctas, G, stream, a)
                   : launch(lp_kernel<E, false, false>, kLpThreads, kLpRing, ctas, G, stream, a);
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
            return shift ? launch(lp_grad_kernel<E, true, true>, kThreads, 0, ctas, 1, stream, a)
                         : launch(lp_grad_kernel<E, true, false>, kThreads, 0, ctas, 1, stream, a);
        return shift ? launch(lp_grad_kernel<E, false, true>, kThreads, 0, ctas, 1, stream, a)
                     : launch(lp_grad_kernel<E, false, false>, kThreads, 0, ctas, 1, stream, a);
    };
    return dtype == SV_BF16 ? typed(__nv_bfloat16()) : typed(0.0f);
}

}  // extern "C"
