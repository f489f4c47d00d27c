// The paged key-value cache of a speculative round: append with rotation,
// attention of the drafted tokens, commit of the accepted ones
// (include/specverify_kv.h).

#include "specverify_kv.h"

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cmath>
#include <cstdint>
#include <mutex>
#include <type_traits>

namespace svkv {

constexpr int kMaxN = 65;       // tree nodes: the root and 64 drafts
constexpr int kMaxDim = 128;
constexpr int kMaxQHeads = 1024;
constexpr int kMaxB = 65535;

// The cache as the kernels see it: byte strides, the page size as a shift.
struct Cache {
    char* k;
    char* v;
    const int32_t* table;
    const float* k_scale;
    const float* v_scale;
    long long page_stride, slot_stride, head_stride;  // bytes
    int num_pages, page_shift, table_width;
    int heads, dim;
};

// ---------------------------------------------------------------- types

template <typename T> struct Conv;
template <> struct Conv<__nv_bfloat16> {
    static __device__ float to(__nv_bfloat16 x) { return __bfloat162float(x); }
    static __device__ __nv_bfloat16 from(float x) { return __float2bfloat16_rn(x); }
};
template <> struct Conv<__half> {
    static __device__ float to(__half x) { return __half2float(x); }
    static __device__ __half from(float x) { return __float2half_rn(x); }
};
template <> struct Conv<__nv_fp8_e4m3> {
    static __device__ float to(__nv_fp8_e4m3 x) { return float(x); }
};

// Two values as a pair of type M in one word (x low), rounded to nearest.
template <typename M> __device__ __forceinline__ uint32_t pair(float x, float y) {
    if constexpr (std::is_same<M, __half>::value) {
        const __half2 h = __floats2half2_rn(x, y);
        return reinterpret_cast<const uint32_t&>(h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        return reinterpret_cast<const uint32_t&>(h);
    }
}
template <typename M> __device__ __forceinline__ float2 unpair(uint32_t w) {
    if constexpr (std::is_same<M, __half>::value)
        return __half22float2(reinterpret_cast<const __half2&>(w));
    else
        return __bfloat1622float2(reinterpret_cast<const __nv_bfloat162&>(w));
}

// V values of a 16-bit type as one access of 2 V bytes (V = 8, 4 or 1), in words.
template <int V> struct Words { uint32_t w[V > 1 ? V / 2 : 1]; };
template <int V> __device__ __forceinline__ Words<V> get(const void* p) {
    Words<V> r;
    if constexpr (V == 8) {
        const uint4 x = *reinterpret_cast<const uint4*>(p);
        r.w[0] = x.x, r.w[1] = x.y, r.w[2] = x.z, r.w[3] = x.w;
    } else if constexpr (V == 4) {
        const uint2 x = *reinterpret_cast<const uint2*>(p);
        r.w[0] = x.x, r.w[1] = x.y;
    } else {
        r.w[0] = *reinterpret_cast<const uint16_t*>(p);
    }
    return r;
}
template <int V> __device__ __forceinline__ void put(void* p, const Words<V>& r) {
    if constexpr (V == 8)
        *reinterpret_cast<uint4*>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    else if constexpr (V == 4)
        *reinterpret_cast<uint2*>(p) = make_uint2(r.w[0], r.w[1]);
    else
        *reinterpret_cast<uint16_t*>(p) = (uint16_t)r.w[0];
}
template <typename T, int V> __device__ __forceinline__ void widen_to(float* f, const Words<V>& r) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
        const float2 x = unpair<T>(r.w[i / 2]);
        f[i] = x.x;
        if (V > 1) f[i + 1] = x.y;
    }
}
// V floats rounded to a 16-bit type and written.
template <typename T, int V> __device__ __forceinline__ void round_to(void* p, const float* f) {
    Words<V> r;
#pragma unroll
    for (int i = 0; i < V; i += 2) r.w[i / 2] = pair<T>(f[i], V > 1 ? f[i + 1] : 0.0f);
    put<V>(p, r);
}
__device__ __forceinline__ uint32_t two_e4m3(float x, float y) {
    return __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
}
// V entries x / scale rounded to float8.  The product with the scale's reciprocal is off by less
// than 2^-22 of itself, and that tells only next to the middle between two float8 values: where the
// ends of an interval of 2^-21 to both sides round alike, that is the entry; the quotients are
// taken where some do not (one element in 2^16), or where the reciprocal is no full float.  (Trees
// of 16 nodes, 64 sequences: 8.2 us, with nothing but quotients 10.2 us.)
template <int V>
__device__ __forceinline__ void put_quotients(void* p, const float* x, float scale) {
    const float inverse = __fdiv_rn(1.0f, scale), size = fabsf(inverse);
    bool near = !(size >= 1e-37f && size <= 3e38f);
    uint32_t w[V > 4 ? 2 : 1] = {};
#pragma unroll
    for (int i = 0; i < V; i += 2) {
        const float u = x[i] * inverse, v = V > 1 ? x[i + 1] * inverse : 0.0f;
        const uint32_t lo = two_e4m3(u * (1.0f - 0x1p-21f), v * (1.0f - 0x1p-21f));
        near |= lo != two_e4m3(u * (1.0f + 0x1p-21f), v * (1.0f + 0x1p-21f));
        w[i / 4] |= lo << (i % 4 * 8);
    }
    if (near) {
        w[0] = w[V > 4 ? 1 : 0] = 0;
#pragma unroll
        for (int i = 0; i < V; ++i)
            w[i / 4] |= (two_e4m3(__fdiv_rn(x[i], scale), 0.0f) & 0xff) << (i % 4 * 8);
    }
    if constexpr (V == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else if constexpr (V == 4) *reinterpret_cast<uint32_t*>(p) = w[0];
    else *reinterpret_cast<uint8_t*>(p) = (uint8_t)w[0];
}

// ---------------------------------------------------------------- sequences

// Whether sequence b's length and number of tokens are good.
__device__ __forceinline__ bool tokens_of(const int32_t* kv_len, const int32_t* num_new, int b,
                                          int N, const Cache& c, int* len, int* n) {
    *n = num_new ? num_new[b] : N;
    *len = kv_len[b];
    const long long cap = (long long)c.table_width << c.page_shift;
    return *n >= 0 && *n <= N && *len >= 0 && (long long)*len + *n <= cap;
}

__device__ __forceinline__ void mark(uint32_t* status, int b, uint32_t bits) {
    if (status) atomicOr(status + b, bits);
}

// Byte offset of slot s of sequence b in k and v, or -1 for a bad page.
__device__ __forceinline__ long long slot_offset(const Cache& c, int b, int s) {
    const int p = __ldg(c.table + (long long)b * c.table_width + (s >> c.page_shift));
    if ((unsigned)p >= (unsigned)c.num_pages) return -1;
    return p * c.page_stride + (s & ((1 << c.page_shift) - 1)) * c.slot_stride;
}

// ---------------------------------------------------------------- append

struct AppendArgs {
    Cache c;
    const uint64_t* turns;
    int rot, interleaved;
    float magnitude;
    const char* q;
    const char* k;
    const char* v;
    char* q_out;
    long long qb, qt, qh, kb, kt, kh;  // elements
    const int32_t* kv_len;
    const int32_t* num_new;
    const int32_t* parents;
    uint32_t* status;
    int N, q_heads, run;  // tokens per CTA
};

constexpr int kAppendThreads = 320;  // at most
constexpr int kAppendHeads = 2;   // heads per thread in flight
constexpr int kAppendTokens = 4;  // at most so many tokens per CTA

// One CTA per run of new tokens of a sequence.  A thread owns the same 2 V elements (V rotated
// pairs, or 2 V elements that are not rotated) of every blockDim.y-th head, queries, keys and
// values in one row.  It asks for its first heads before anything else; the lengths, the pages
// and the angles of the run arrive while they are under way, and each next token's heads while
// the one before is turned and written.  The angle is position * rate modulo one turn in 64-bit
// integers (exact), so far positions lose nothing; its top 32 bits become the argument of
// sincospi.  Accesses are of 16 bytes where V = 8.  Bound by memory: each query, key and value is
// read once and written once (256 x 65 tokens of 80 heads of 128: 119 us, 5.7 TB/s).
template <typename T, typename CT, int V, bool INTERLEAVED>
__global__ void __launch_bounds__(kAppendThreads, 2) kv_append_kernel(const AppendArgs a) {
    __shared__ float2 s_cs[kAppendTokens][kMaxDim / 2];
    __shared__ long long s_place[kAppendTokens];
    __shared__ int s_par[kMaxN];
    const int b = blockIdx.y, j0 = blockIdx.x * a.run, w = threadIdx.x;
    const int tid = threadIdx.y * blockDim.x + w, threads = blockDim.x * blockDim.y;
    const Cache& c = a.c;
    struct Heads { Words<V> x0[kAppendHeads], x1[kAppendHeads]; };
    const int half = a.rot / 2, D = c.dim, qn = a.q ? a.q_heads : 0, heads = qn + 2 * c.heads;
    const bool turns = w < half / V;
    const int e0 = turns && !INTERLEAVED ? w * V : 2 * w * V;
    const int e1 = turns && !INTERLEAVED ? e0 + half : e0 + V;
    auto load = [&](Heads& x, int j, int h0) {
#pragma unroll
        for (int i = 0; i < kAppendHeads; ++i) {
            const int h = h0 + i * blockDim.y;
            if (h >= heads) continue;
            const T* src = h < qn ? (const T*)a.q + b * a.qb + j * a.qt + h * a.qh
                           : h < qn + c.heads
                               ? (const T*)a.k + b * a.kb + j * a.kt + (h - qn) * a.kh
                               : (const T*)a.v + b * a.kb + j * a.kt + (h - qn - c.heads) * a.kh;
            x.x0[i] = get<V>(src + e0);
            x.x1[i] = get<V>(src + e1);
        }
    };
    Heads now, next;
    load(now, j0, threadIdx.y);

    int len, n;
    if (!tokens_of(a.kv_len, a.num_new, b, a.N, c, &len, &n)) {
        if (j0 == 0 && tid == 0) mark(a.status, b, SV_DEV_BAD_LENGTH);
        return;
    }
    const int j1 = min(n, j0 + a.run);
    if (j0 >= j1) return;
    // (a block of one or two short heads has fewer threads than its run has tokens)
    for (int i = tid; i < j1 - j0; i += threads) {
        s_place[i] = slot_offset(c, b, len + j0 + i);
        if (s_place[i] < 0) mark(a.status, b, SV_DEV_BAD_PAGE);
    }
    if (a.parents) {
        int bad = 0;
        for (int i = tid; i < n; i += threads) {
            const int p = a.parents[(long long)b * a.N + i];
            s_par[i] = p;
            bad |= i > 0 && (p < 0 || p >= i);
        }
        if (__syncthreads_or(bad)) {
            if (j0 == 0 && tid == 0) mark(a.status, b, SV_DEV_BAD_TREE);
            return;
        }
    }
    for (int i = tid; i < half * (j1 - j0); i += threads) {
        const int t = i / half, e = i - t * half;
        int depth = j0 + t;
        if (a.parents) {
            depth = 0;
            for (int k = j0 + t; k > 0; k = s_par[k]) ++depth;
        }
        const int32_t turn = (int32_t)((((uint64_t)len + depth) * a.turns[e]) >> 32);
        float s, co;
        sincospif((float)turn * 4.656612873077393e-10f, &s, &co);  // 2^-31: half turns
        s_cs[t][e] = make_float2(co * a.magnitude, s * a.magnitude);
    }
    __syncthreads();

    auto write = [&](const Heads& x, int j, int h0) {
        const long long place = s_place[j - j0];
        float2 cs[V];
#pragma unroll
        for (int i = 0; i < V; ++i)
            cs[i] = turns ? s_cs[j - j0][w * V + i] : make_float2(1.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < kAppendHeads; ++i) {
            const int h = h0 + i * blockDim.y;
            if (h >= heads) continue;
            const bool is_q = h < qn, is_v = h >= qn + c.heads;
            const int ch = is_v ? h - qn - c.heads : h - qn;  // head of the cache
            if (!is_q && place < 0) continue;
            if (is_v && sizeof(CT) == sizeof(T)) {  // moved bit by bit
                CT* dst = (CT*)(c.v + place + ch * c.head_stride);
                put<V>(dst + e0, x.x0[i]);
                put<V>(dst + e1, x.x1[i]);
                continue;
            }
            float r[2 * V];
            widen_to<T, V>(r, x.x0[i]);
            widen_to<T, V>(r + V, x.x1[i]);
            if (turns && !is_v) {
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    // the pair's places among the thread's 2 V elements
                    float& u = r[INTERLEAVED ? 2 * k : k];
                    float& v = r[INTERLEAVED ? 2 * k + 1 : V + k];
                    const float p = u * cs[k].x - v * cs[k].y;
                    v = v * cs[k].x + u * cs[k].y;
                    u = p;
                }
            }
            if (is_q) {
                T* dst = (T*)a.q_out + (((long long)b * a.N + j) * a.q_heads + h) * D;
                round_to<T, V>(dst + e0, r);
                round_to<T, V>(dst + e1, r + V);
            } else {
                CT* dst = (CT*)((is_v ? c.v : c.k) + place + ch * c.head_stride);
                if constexpr (sizeof(CT) == 1) {
                    const float scale = (is_v ? c.v_scale : c.k_scale)[ch];
                    put_quotients<V>(dst + e0, r, scale);
                    put_quotients<V>(dst + e1, r + V, scale);
                } else {
                    round_to<CT, V>(dst + e0, r);
                    round_to<CT, V>(dst + e1, r + V);
                }
            }
        }
    };
    for (int j = j0; j < j1; ++j) {
        if (j + 1 < j1) load(next, j + 1, threadIdx.y);
        write(now, j, threadIdx.y);
        for (int h0 = threadIdx.y + kAppendHeads * blockDim.y; h0 < heads;
             h0 += kAppendHeads * blockDim.y) {
            load(now, j, h0);
            write(now, j, h0);
        }
        now = next;
    }
}

// ---------------------------------------------------------------- attention
//
// out_j = sum_l p_jl v_l, p_j = softmax over the visible slots l of scale * q_j . k_l.
//
// The query rows of one key head (new token j, group member g: row j * group + g) are the rows
// of a matrix product with the keys, so that a key or value is read from memory once for all of
// them.  Work is cut by bytes, not by sequences: an item is (sequence, key head, row tile), it
// has one unit per 64 slots, and the units of all items, in order, are cut into one equal range
// per resident CTA, whatever the lengths (they are known on the device only).  A CTA whose range
// ends inside an item leaves its running maximum, sum and output in the workspace (at most two
// such pieces per CTA), and the join kernel adds the pieces of an item up.  Which CTA does what
// depends on the lengths alone, so results repeat bit for bit.

struct AttentionArgs {
    Cache c;
    const char* q;
    char* out;
    long long qb, qt, qh;  // elements
    const int32_t* kv_len;
    const int32_t* num_new;
    const int32_t* parents;
    uint32_t* status;
    float scale;
    int B, N, q_heads, group;
    int ctas;             // ranges
    int mts;              // row tiles of an item's head, counted for N tokens
    int* started;         // workspace: [ctas] the item that a range starts and another goes on
                          // with, or -1: there is at most one, its last
    int* ended;           // workspace: [B, heads, mts] the range that ends an item begun by another
    float* part_o;        // workspace: [2 * ctas, rows, DP], or of the wide kernel
                          // [2 * ctas, DP / 4, rows, 4]: there a thread holds a row
    float2* part_ml;      // workspace: [2 * ctas, rows] maximum (base 2) and sum
};

constexpr int kUnit = 64;          // slots of a unit: 16 per warp
constexpr int kSplitThreads = 128;
constexpr int kMaxCtas = 304;      // two per SM

// One sequence's share of the work, for row tiles of `rows` rows.  A unit of a tile of 256 rows
// weighs as two where more than 128 of them are there: it takes both streams' time.
struct Share {
    int len, n, tiles, mts;
    int last;  // weight of the last row tile's units; the others weigh `full`
    bool bad;
    __device__ long long units(int heads, int full) const {
        return (long long)heads * tiles * (mts > 0 ? full * (mts - 1) + last : 0);
    }
};
__device__ __forceinline__ constexpr int full_weight(int rows) { return rows > 128 ? 2 : 1; }

__device__ __forceinline__ Share share_of(const AttentionArgs& a, int b, int rows, int unit) {
    Share s;
    s.bad = !tokens_of(a.kv_len, a.num_new, b, a.N, a.c, &s.len, &s.n);
    // one unit per item of a bad one: its rows become NaN, all N where the count itself is bad
    if (s.n < 0 || s.n > a.N) s.n = a.N;
    s.tiles = s.bad ? 1 : (int)(((long long)s.len + s.n + unit - 1) / unit);
    s.mts = (s.n * a.group + rows - 1) / rows;
    s.last = s.n * a.group - (s.mts - 1) * rows > 128 ? 2 : 1;
    return s;
}

// Ranges that units of total weight W are cut into: each has a whole unit at least.
__device__ __forceinline__ int ranges_of(long long W, int ctas, int full) {
    return (int)min((long long)ctas, max(W / full, 1ll));
}
// Range c of P equal ranges of W units starts at floor(c W / P).
__device__ __forceinline__ long long range_start(long long W, int P, int c) {
    return W / P * c + W % P * c / P;
}

// A CTA's range as pieces of items, in order: sequence, key head, row tile, units t0 .. t1 - 1.
struct Piece {
    int b, h, mt, t0, t1, rows;
};
struct Walk {
    long long left;  // weight of the range still to come
    long long at;    // weight of the item before the range's part of it
    int b, item;
    Share sh;
    __device__ __forceinline__ bool next(const AttentionArgs& a, int rows, int unit, Piece* p) {
        const int full = full_weight(rows);
        for (;;) {
            if (left <= 0) return false;
            while (item >= a.c.heads * sh.mts) {
                sh = share_of(a, ++b, rows, unit);
                item = 0;
            }
            p->b = b;
            p->h = item / sh.mts;
            p->mt = item - p->h * sh.mts;
            // (a unit of weight two belongs to the range that its first half is in)
            const int w = full == 1 || p->mt < sh.mts - 1 ? full : sh.last;
            const long long to = min((long long)sh.tiles * w, at + left);
            p->t0 = (int)((at + w - 1) / w);
            p->t1 = (int)((to + w - 1) / w);
            p->rows = min(rows, sh.n * a.group - p->mt * rows);
            left -= to - at;
            ++item;
            at = 0;
            if (p->t0 < p->t1) return true;
        }
    }
};
struct Start {
    long long at;
    int b;
};

// Says where the pieces of an item are, for the join.
__device__ __forceinline__ void tell_ends(const AttentionArgs& a, const Piece& p, int tiles) {
    const int item = (p.b * a.c.heads + p.h) * a.mts + p.mt;
    if (p.t0 == 0 && p.t1 < tiles) a.started[blockIdx.x] = item;
    if (p.t0 > 0 && p.t1 == tiles) a.ended[item] = blockIdx.x;
}

// The range of this CTA: weight of the units before each sequence (a scan over the batch), their
// sum W, range blockIdx.x of those that W is cut into.
template <int THREADS>
__device__ __forceinline__ Walk start_walk(const AttentionArgs& a, int rows, int unit,
                                           long long* s_scan, Start* s_start) {
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, full = full_weight(rows);
    const int per = (a.B + THREADS - 1) / THREADS;
    const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    long long sum = 0;
    for (int b = b0; b < b1; ++b) {
        const Share s = share_of(a, b, rows, unit);
        sum += s.units(a.c.heads, full);
        // (here: a sequence without tokens has no piece that would say so)
        if (s.bad && blockIdx.x == 0) mark(a.status, b, SV_DEV_BAD_LENGTH);
    }
    long long inc = sum;
    for (int k = 1; k < 32; k <<= 1) {
        const long long y = __shfl_up_sync(~0u, inc, k);
        if (lane >= k) inc += y;
    }
    if (lane == 31) s_scan[w] = inc;
    __syncthreads();
    long long W = 0, before = inc - sum;
    for (int i = 0; i < THREADS / 32; ++i) {
        W += s_scan[i];
        if (i < w) before += s_scan[i];
    }
    if (tid == 0) a.started[blockIdx.x] = -1;  // until it starts one that it does not end
    const int P = ranges_of(W, a.ctas, full);
    const bool some = W > 0 && (int)blockIdx.x < P;
    const long long x = some ? range_start(W, P, blockIdx.x) : 0;
    const bool here = some && x >= before && x < before + sum;
    if (here) {
        long long at = before;
        for (int b = b0; b < b1; ++b) {
            const long long u = share_of(a, b, rows, unit).units(a.c.heads, full);
            if (x >= at && x < at + u) *s_start = Start{at, b};
            at += u;
        }
    }
    __syncthreads();
    Walk k = {};
    if (some) {
        k.left = range_start(W, P, blockIdx.x + 1) - x;
        k.b = s_start->b;
        k.sh = share_of(a, k.b, rows, unit);
        const long long r = x - s_start->at, head = k.sh.units(1, full);
        const long long tile = (long long)k.sh.tiles * full;  // weight of an item but the last
        const int h = (int)(r / head);
        const int mt = (int)min((r - h * head) / tile, (long long)k.sh.mts - 1);
        k.item = h * k.sh.mts + mt;
        k.at = r - h * head - mt * tile;
    }
    return k;
}

// Clusters of CTAs, one per item.
constexpr int kCluster = 8;
__device__ __forceinline__ int cluster_rank() {
    int r;
    asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
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
// The part of its cluster's item that this CTA takes: equal shares of the units, perhaps none.
// False for an item that the sequence does not have (fewer tokens than the launch counts on).
__device__ __forceinline__ bool item_piece(const AttentionArgs& a, int rows, int unit, Share* sh,
                                           Piece* p) {
    const int mts = (a.N * a.group + rows - 1) / rows, item = blockIdx.x / kCluster;
    p->mt = item % mts;
    p->h = item / mts % a.c.heads;
    p->b = item / mts / a.c.heads;
    *sh = share_of(a, p->b, rows, unit);
    const int rank = cluster_rank();
    if (sh->bad && p->mt == 0 && rank == 0 && threadIdx.x == 0)
        mark(a.status, p->b, SV_DEV_BAD_LENGTH);
    if (p->mt >= sh->mts) return false;
    p->t0 = (int)((long long)sh->tiles * rank / kCluster);
    p->t1 = (int)((long long)sh->tiles * (rank + 1) / kCluster);
    p->rows = min(rows, sh->n * a.group - p->mt * rows);
    return true;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool take) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(take ? 16 : 0));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
template <typename M>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
    if constexpr (sizeof(M) == 2 && !std::is_same<M, __half>::value)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, "
                     "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, "
                     "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The high half of a pair that a low half will make up for: bf16 by leaving off bits.
template <typename M> __device__ __forceinline__ uint32_t cut(float x, float y) {
    if constexpr (std::is_same<M, __half>::value) return pair<M>(x, y);
    else return __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{ .reg .b64 a, b, c; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mov.b64 c, {%6, %7}; "
        "fma.rn.f32x2 a, a, b, c; mov.b64 {%0, %1}, a; }"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{ .reg .b64 a, b; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; "
        "add.rn.f32x2 a, a, b; mov.b64 {%0, %1}, a; }"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
// Four e4m3 bytes as two pairs of halves (bytes 0 and 1, bytes 2 and 3): exact.
__device__ __forceinline__ void widen(uint32_t& low, uint32_t& high, uint32_t w) {
    asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; "
        "cvt.rn.f16x2.e4m3x2 %1, h; }" : "=r"(low), "=r"(high) : "r"(w));
}

// The power of two that a query row of bfloat16 is divided by to fit halves, top its largest
// element: at most 119 (2^127), at least -126, so that 2^-e and 2^e are floats.  It is multiplied
// back before the key scale, which may be as small as the row is large.
__device__ __forceinline__ int row_power(float top) {
    return top > 0.0f && top < INFINITY ? max(-126, ilogbf(top) - 8) : 0;
}

// Layout of a warp's stage: 16 keys, then 16 values, rows of DP elements whose 16-byte chunks
// are exchanged so that neither ldmatrix (8 rows, one chunk) nor the 16-byte loads of float8
// keys (two rows, four chunks at a time) meet in a bank.
template <typename CT, int DP> struct Stage {
    static constexpr int kPitch = DP * (int)sizeof(CT);
    static constexpr int kChunks = kPitch / 16;  // 4, 8 or 16
    static constexpr int kBytes = 2 * 16 * kPitch;
    // as many stages as fit 96 KiB for the four warps (two CTAs per SM), six at most
    static constexpr int kStages = 4 * kBytes * 6 <= 98304 ? 6 : 98304 / (4 * kBytes);
    static __device__ __forceinline__ int at(int row, int chunk) {
        const int x = kChunks == 16  ? chunk ^ (row & 7)
                      : kChunks == 8 ? chunk ^ ((row & 1) << 2 | (row >> 1 & 3))
                                     : chunk ^ (row >> 1 & 3);
        return row * kPitch + x * 16;
    }
};

// Whether node j's row may look at new token i of the sequence (bit i - 1 of its ancestors).
__device__ __forceinline__ bool sees(uint64_t anc, int i) { return i == 0 || (anc >> (i - 1) & 1); }

// Rows of a CTA: WM * 16, at most 32.  Each of the four slot groups walks its own 16 slots of
// every unit, with its own ring of stages filled by 16-byte asynchronous copies; in it a warp per
// 16 rows keeps its own running maximum, sum and output (one warp: no barrier inside a piece; two
// share the ring and meet once per stage, and keep their queries in shared memory, so that 16
// warps fit an SM).  The four groups are joined in shared memory at a piece's end.  Matrix
// products by mma.sync: with at most 32 rows the tensor pipe has time to spare, and the weights
// may take two products: P = hi + lo, two 16-bit halves, so that rounding the weights costs
// nothing next to rounding the result.  float8 caches become halves on the way into the registers
// (exact), with a power of two taken out of each query row so that a bfloat16 query fits a half
// too; their weights are single halves then, three bits finer than a bfloat16 result (fewer below
// 2^-14 of the reference).  Bound by memory up to 16 rows (64 sequences of 4000-8000 slots, one
// token, 32 query and 8 key heads of 128: 246 us, 6.4 TB/s; the same over float8, 96 sequences of
// 4100-8200 slots: 223 us, 5.5 TB/s), by conversions and fixed latencies over float8 with 32 (96
// sequences, 24 rows: 353 us, 3.5 TB/s).
template <typename CT, int DP, int WM> struct Split {
    using St = Stage<CT, DP>;
    static constexpr int kRows = WM * 16, kPitch = DP + 8;  // floats: rows eight banks apart
    static constexpr int kRing = 4 * St::kStages * St::kBytes;
    static constexpr int kMerge = 4 * kRows * kPitch * 4 + 4 * kRows * 8;
    static constexpr int kShare = kRows * DP * 4 + kRows * 8;  // a cluster's CTA's own sums
    static constexpr int kBody = kRing > kMerge + kShare ? kRing : kMerge + kShare;
    static constexpr int kSmem = kBody + (WM > 1 ? kRows * DP * 2 : 0);  // + queries
};

//
// CLUSTER: a cluster of kCluster CTAs per item instead, each with an equal share of its units,
// joined through distributed shared memory: one launch and no workspace, for calls of few items
// and short contexts, whose time is latency (one sequence of 700 positions: 8.4 us with the join
// kernel, 5.6 us so).
template <typename T, typename CT, int DP, int WM, bool CLUSTER>
__global__ void __launch_bounds__(kSplitThreads * WM, 2) kv_split_kernel(const AttentionArgs a) {
    constexpr bool kF8 = sizeof(CT) == 1;
    using M = typename std::conditional<kF8, __half, T>::type;  // type of the products
    constexpr bool kFit = !kF8 || std::is_same<T, __half>::value;  // queries are of it already
    constexpr bool kLo = kFit;
    using St = Stage<CT, DP>;
    using L = Split<CT, DP, WM>;
    constexpr int S = St::kStages, KS = DP / 16, NT = DP / 8, ROWS = L::kRows;
    constexpr int THREADS = kSplitThreads * WM;
    extern __shared__ __align__(128) char smem[];
    __shared__ long long s_scan[THREADS / 32];
    __shared__ Start s_start;
    __shared__ int s_par[kMaxN];
    __shared__ uint64_t s_anc[kMaxN];
    const int tid = threadIdx.x, lane = tid & 31, t4 = lane & 3;
    const int w = tid >> 5 & 3, wm = tid >> 7;  // slot group, row tile
    const Cache& c = a.c;
    auto group_sync = [&]() {
        if constexpr (WM == 1)
            __syncwarp();
        else
            asm volatile("bar.sync %0, %1;" ::"r"(1 + w), "r"(32 * WM) : "memory");
    };

    cudaGridDependencySynchronize();
    cudaTriggerProgrammaticLaunchCompletion();

    Walk walk = {};
    if constexpr (!CLUSTER) walk = start_walk<THREADS>(a, ROWS, kUnit, s_scan, &s_start);
    const Share& sh = walk.sh;
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(smem);
    const uint32_t ring = base + w * S * St::kBytes;
    const uint32_t queries = base + L::kBody + wm * KS * 512 + lane * 16;
    int anc_of = -1;  // the sequence whose ancestors s_anc holds

    Piece piece;
    while (CLUSTER ? item_piece(a, ROWS, kUnit, &walk.sh, &piece)
                   : walk.next(a, ROWS, kUnit, &piece)) {
        const int b = piece.b, h = piece.h, mt = piece.mt, t0 = piece.t0, t1 = piece.t1;
        const int len = sh.len, total = len + sh.n, rows = piece.rows;
        if (!CLUSTER && tid == 0) tell_ends(a, piece, sh.tiles);
        bool bad = sh.bad;

        const char* kb = c.k + h * c.head_stride;
        const char* vb = c.v + h * c.head_stride;
        const int32_t* table = c.table + (long long)b * c.table_width;
        const int my = w * 16 + (lane & 15);  // the slot of a unit whose page this lane looks up
        const int dch = c.dim * (int)sizeof(CT) / 16;
        bool bad_page = false;
        auto page_of = [&](int t) -> int {
            const int s = t * kUnit + my;
            return t < t1 && s < total ? __ldg(table + (s >> c.page_shift)) : -1;
        };
        auto issue = [&](int t, int stage, int page) {
            const int s = t * kUnit + my;
            long long off = -1;
            if (t < t1 && s < total) {
                if ((unsigned)page < (unsigned)c.num_pages)
                    off = page * c.page_stride + (s & ((1 << c.page_shift) - 1)) * c.slot_stride;
                else
                    bad_page = true;
            }
            if (t < t1) {
                const uint32_t dst = ring + stage * St::kBytes;
                constexpr int kRows = 32 / St::kChunks;  // rows per instruction
                constexpr int kMine = 16 / kRows / WM;
#pragma unroll
                for (int i = 0; i < kMine; ++i) {
                    const int row = (i * WM + wm) * kRows + lane / St::kChunks;
                    const int ch = lane % St::kChunks;
                    const long long f = __shfl_sync(~0u, off, row);
                    const bool take = f >= 0 && ch < dch;
                    const long long at = take ? f + ch * 16 : 0;
                    cp_async16(dst + St::at(row, ch), kb + at, take);
                    cp_async16(dst + 16 * St::kPitch + St::at(row, ch), vb + at, take);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        int page = -1;
        if (!bad) {
            int first[S - 1];
#pragma unroll
            for (int i = 0; i < S - 1; ++i) first[i] = page_of(t0 + i);
            page = page_of(t0 + S - 1);
#pragma unroll
            for (int i = 0; i < S - 1; ++i) issue(t0 + i, i, first[i]);
        }

        // With the first slots on their way: the ancestors of every node, where this piece reaches
        // the new tokens.
        if (!bad && (long long)t1 * kUnit > len && anc_of != b) {
            __syncthreads();
            int f = 0;
            if (a.parents)
                for (int i = tid; i < sh.n; i += THREADS) {
                    const int p = a.parents[(long long)b * a.N + i];
                    s_par[i] = p;
                    f |= i > 0 && (p < 0 || p >= i);
                }
            f = __syncthreads_or(f);
            if (tid < sh.n) {
                uint64_t m = 0;
                if (!a.parents)
                    m = tid == 64 ? ~0ull : (1ull << tid) - 1;
                else if (!f)
                    for (int i = tid; i > 0; i = s_par[i]) m |= 1ull << (i - 1);
                s_anc[tid] = m;
            }
            __syncthreads();
            if (f) {
                bad = true;
                if (tid == 0) mark(a.status, b, SV_DEV_BAD_TREE);
                anc_of = -1;
            } else {
                anc_of = b;
            }
        }

        // Queries as the A operand: thread (row lane / 4, + 8; elements by lane % 4), with the
        // sign of the scales, so that the largest product is the largest exponent.
        uint32_t qa[KS][4];
        float mul[2];  // from a product to the exponent (base 2)
        const float ks_h = kF8 ? c.k_scale[h] : 1.0f;
        const float unit = fabsf(a.scale) * 1.4426950408889634f * fabsf(ks_h);
        const uint32_t sign = (a.scale < 0.0f) != (ks_h < 0.0f) ? 0x80008000u : 0u;
        // never 0, for 0 * -inf is NaN; a scale that is NaN stays so
        auto not_zero = [](float x) { return x < 1e-37f ? 1e-37f : x; };
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int row = wm * 16 + half * 8 + (lane >> 2), R = mt * ROWS + row;
            const int j = R / a.group, g = R - j * a.group;
            const bool live = row < rows && !bad;
            const T* q = (const T*)a.q + (live ? b * a.qb + j * a.qt +
                                                     (long long)(h * a.group + g) * a.qh : 0);
            float top = 0.0f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                // float8: 16 consecutive elements of a block of 64 per thread, 4 per step
                const int e0 = kF8 ? (ks >> 2) * 64 + t4 * 16 + (ks & 3) * 4 : ks * 16 + t4 * 2;
                const int e1 = kF8 ? e0 + 2 : e0 + 8;
                const bool in = live && (kF8 ? e0 : ks * 16) < c.dim;
                const uint32_t w0 = in ? __ldg((const uint32_t*)(q + e0)) ^ sign : 0u;
                const uint32_t w1 = in ? __ldg((const uint32_t*)(q + e1)) ^ sign : 0u;
                qa[ks][half] = w0;
                qa[ks][half + 2] = w1;
                if constexpr (!kFit) {
                    const float2 f0 = unpair<T>(w0), f1 = unpair<T>(w1);
                    top = fmaxf(fmaxf(top, fmaxf(fabsf(f0.x), fabsf(f0.y))),
                                fmaxf(fabsf(f1.x), fabsf(f1.y)));
                }
            }
            mul[half] = not_zero(unit);
            if constexpr (!kFit) {
                top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
                top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
                // the row's largest element becomes 2^8 .. 2^9: what then falls below the smallest
                // half is 2^-33 of it
                const int e = row_power(top);
                const float down = exp2f((float)-e);
                mul[half] = not_zero(fabsf(a.scale) * 1.4426950408889634f * exp2f((float)e) *
                                     fabsf(ks_h));
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int k = half; k < 4; k += 2) {
                        const float2 f = unpair<T>(qa[ks][k]);
                        qa[ks][k] = pair<__half>(f.x * down, f.y * down);
                    }
            }
        }
        if constexpr (WM > 1) {  // kept in shared memory, as each lane will want them
            if (w == 0)
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
                    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(queries + ks * 512),
                                 "r"(qa[ks][0]), "r"(qa[ks][1]), "r"(qa[ks][2]), "r"(qa[ks][3])
                                 : "memory");
            __syncthreads();
        }
        auto query = [&](int ks, uint32_t (&f)[4]) {
            if constexpr (WM > 1)
                asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                             : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3])
                             : "r"(queries + ks * 512) : "memory");
            else
                for (int k = 0; k < 4; ++k) f[k] = qa[ks][k];
        };

        float o[NT][4], l[2] = {0.0f, 0.0f}, mr[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < NT; ++k) o[k][0] = o[k][1] = o[k][2] = o[k][3] = 0.0f;

        int stage = 0;
        for (int t = t0; t < t1 && !bad; ++t) {
            asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
            group_sync();
            issue(t + S - 1, stage == 0 ? S - 1 : stage - 1, page);
            page = page_of(t + S);
            const uint32_t kt = ring + stage * St::kBytes, vt = kt + 16 * St::kPitch;
            stage = stage == S - 1 ? 0 : stage + 1;
            const int slot0 = t * kUnit + w * 16;
            if (slot0 >= total) continue;

            // Scores: 16 slots = two tiles of 8 columns.
            float s[2][4];
#pragma unroll
            for (int k = 0; k < 4; ++k) s[0][k] = s[1][k] = 0.0f;
            if constexpr (!kF8) {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    uint32_t f[4], q[4];
                    const int row = (lane & 7) + (lane >> 4) * 8, ch = ks * 2 + (lane >> 3 & 1);
                    ldsm4(f, kt + St::at(row, ch));
                    query(ks, q);
                    mma<M>(s[0], q, f[0], f[1]);
                    mma<M>(s[1], q, f[2], f[3]);
                }
            } else {
#pragma unroll
                for (int kb4 = 0; kb4 < DP / 64; ++kb4) {
                    uint32_t f[2][4];
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt)
                        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                                     : "=r"(f[nt][0]), "=r"(f[nt][1]), "=r"(f[nt][2]),
                                       "=r"(f[nt][3])
                                     : "r"(kt + St::at(nt * 8 + (lane >> 2), kb4 * 4 + t4))
                                     : "memory");
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t q[4];
                        query(kb4 * 4 + k, q);
#pragma unroll
                        for (int nt = 0; nt < 2; ++nt) {
                            uint32_t b0, b1;
                            widen(b0, b1, f[nt][k]);
                            mma<M>(s[nt], q, b0, b1);
                        }
                    }
                }
            }
            const bool fresh = slot0 > len - 16;  // new tokens or the end are among the 16
            if (fresh) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int R = mt * ROWS + wm * 16 + half * 8 + (lane >> 2);
                    const uint64_t anc = s_anc[min(R / a.group, sh.n - 1)];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int i = slot0 + (k >> 1) * 8 + t4 * 2 + (k & 1) - len;
                        if (i >= 0 && (i >= sh.n || !sees(anc, i)))
                            s[k >> 1][half * 2 + (k & 1)] = -INFINITY;
                    }
                }
            }
            // The reference of a row follows its maximum only when that has grown by 2^8: weights
            // stay below 2^8 and the output is rarely rescaled.
            float mx[2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float m = fmaxf(fmaxf(s[0][half * 2], s[0][half * 2 + 1]),
                                fmaxf(s[1][half * 2], s[1][half * 2 + 1]));
                m = fmaxf(m, __shfl_xor_sync(~0u, m, 1));
                m = fmaxf(m, __shfl_xor_sync(~0u, m, 2));
                mx[half] = m * mul[half];
            }
            const bool grow0 = mx[0] > mr[0] + 8.0f, grow1 = mx[1] > mr[1] + 8.0f;
            if (__any_sync(~0u, grow0 || grow1)) {
                const float f0 = grow0 ? ex2(mr[0] - mx[0]) : 1.0f;
                const float f1 = grow1 ? ex2(mr[1] - mx[1]) : 1.0f;
                if (grow0) mr[0] = mx[0];
                if (grow1) mr[1] = mx[1];
                l[0] *= f0;
                l[1] *= f1;
#pragma unroll
                for (int k = 0; k < NT; ++k) {
                    o[k][0] *= f0;
                    o[k][1] *= f0;
                    o[k][2] *= f1;
                    o[k][3] *= f1;
                }
            }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const float ref = mr[half] == -INFINITY ? 0.0f : mr[half];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float& p = s[k >> 1][half * 2 + (k & 1)];
                    p = ex2(fmaf(p, mul[half], -ref));
                    l[half] += p;
                }
            }
            if (fresh) {
                // A masked entry may hold anything, but 0 times NaN is NaN: values that are not
                // finite are taken out of the product and added for the rows that see them.
                bool f = false;
                const int row = lane >> 1;
                if (slot0 + row > len && slot0 + row < total) {
                    for (int ch = (lane & 1); ch < dch; ch += 2) {
                        uint32_t v[4];
                        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                                     : "r"(vt + St::at(row, ch)) : "memory");
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if constexpr (kF8) {
                                for (int i = 0; i < 32; i += 8) f |= (v[k] >> i & 0x7f) == 0x7f;
                            } else {
                                constexpr uint32_t e = std::is_same<T, __half>::value ? 0x7c00u
                                                                                      : 0x7f80u;
                                f |= (v[k] & e) == e || (v[k] >> 16 & e) == e;
                            }
                        }
                    }
                }
                const uint32_t wild = __ballot_sync(~0u, f);  // (the same in the group's warps)
                for (int rw = 0; wild != 0 && rw < 16; ++rw) {
                    if (!(wild >> (2 * rw) & 3)) continue;
                    const int i = slot0 + rw - len;
                    const int from = (lane & ~3) | (rw & 7) >> 1;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const float pe = rw < 8 ? s[0][half * 2] : s[1][half * 2];
                        const float po = rw < 8 ? s[0][half * 2 + 1] : s[1][half * 2 + 1];
                        const float p = __shfl_sync(~0u, rw & 1 ? po : pe, from);
                        const int R = mt * ROWS + wm * 16 + half * 8 + (lane >> 2);
                        if (sees(s_anc[min(R / a.group, sh.n - 1)], i)) {
#pragma unroll
                            for (int k = 0; k < NT; ++k)
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const int d = kF8 ? (k >> 1) * 16 + t4 * 4 + e * 2 + (k & 1)
                                                      : k * 8 + t4 * 2 + e;
                                    const int by = d * (int)sizeof(CT);
                                    const CT* v = reinterpret_cast<const CT*>(
                                        smem + (vt + St::at(rw, by >> 4) + (by & 15) - base));
                                    o[k][half * 2 + e] += p * Conv<CT>::to(*v);
                                }
                        }
                        __syncwarp();
                    }
                }
                if (wild) {
                    group_sync();  // every warp of the group has added its own
                    for (int rw = 0; rw < 16; ++rw)
                        if (wild >> (2 * rw) & 3)
                            for (int ch = lane; ch < St::kChunks; ch += 32)
                                asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(
                                                 vt + St::at(rw, ch)), "r"(0) : "memory");
                    group_sync();
                }
            }
            uint32_t pa[4], pl[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float u = s[k >> 1][(k & 1) * 2], v = s[k >> 1][(k & 1) * 2 + 1];
                if constexpr (kLo) {
                    pa[k] = cut<M>(u, v);
                    const float2 f = unpair<M>(pa[k]);
                    pl[k] = pair<M>(u - f.x, v - f.y);
                } else {
                    pa[k] = pair<M>(u, v);
                }
            }
            if constexpr (!kF8) {
#pragma unroll
                for (int dt = 0; dt < KS; ++dt) {
                    uint32_t f[4];
                    ldsm4t(f, vt + St::at(lane & 15, dt * 2 + (lane >> 4)));
                    mma<M>(o[2 * dt], pa, f[0], f[1]);
                    mma<M>(o[2 * dt + 1], pa, f[2], f[3]);
                    mma<M>(o[2 * dt], pl, f[0], f[1]);
                    mma<M>(o[2 * dt + 1], pl, f[2], f[3]);
                }
            } else {
                // a word: elements 2i and 2i + 1 of two slots; the even elements make one tile of
                // 8 columns, the odd ones the next
#pragma unroll
                for (int dt = 0; dt < DP / 32; ++dt) {
                    uint32_t f[4];
                    ldsm4t(f, vt + St::at(lane & 15, dt * 2 + (lane >> 4)));
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t e0, e1, o0, o1;
                        widen(e0, o0, __byte_perm(f[2 * k], 0, 0x3120));
                        widen(e1, o1, __byte_perm(f[2 * k + 1], 0, 0x3120));
                        mma<M>(o[4 * dt + 2 * k], pa, e0, e1);
                        mma<M>(o[4 * dt + 2 * k + 1], pa, o0, o1);
                        if constexpr (kLo) {
                            mma<M>(o[4 * dt + 2 * k], pl, e0, e1);
                            mma<M>(o[4 * dt + 2 * k + 1], pl, o0, o1);
                        }
                    }
                }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        bad_page = __syncthreads_or(bad_page);
        if (bad_page) {
            if (tid == 0) mark(a.status, b, SV_DEV_BAD_PAGE);
            bad = true;
        }

        // Join the four groups.
        float* so = reinterpret_cast<float*>(smem);
        constexpr int kP = L::kPitch;
        float2* sml = reinterpret_cast<float2*>(so + 4 * ROWS * kP);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int row = wm * 16 + half * 8 + (lane >> 2);
            float sum = l[half];
            sum += __shfl_xor_sync(~0u, sum, 1);
            sum += __shfl_xor_sync(~0u, sum, 2);
            if (t4 == 0) sml[w * ROWS + row] = make_float2(mr[half], sum);
            float* dst = so + (w * ROWS + row) * kP;
            if constexpr (!kF8) {
#pragma unroll
                for (int k = 0; k < NT; ++k)
                    *reinterpret_cast<float2*>(dst + k * 8 + t4 * 2) =
                        make_float2(o[k][half * 2], o[k][half * 2 + 1]);
            } else {
#pragma unroll
                for (int k = 0; k < NT; k += 2)
                    *reinterpret_cast<float4*>(dst + k * 8 + t4 * 4) =
                        make_float4(o[k][half * 2], o[k + 1][half * 2], o[k][half * 2 + 1],
                                    o[k + 1][half * 2 + 1]);
            }
        }
        __syncthreads();
        const bool whole = !CLUSTER && t0 == 0 && t1 == sh.tiles;
        const long long part = 2 * blockIdx.x + (t0 == 0 ? 1 : 0);
        const float vs = kF8 ? c.v_scale[h] : 1.0f;
        // (cluster: this CTA's share, behind what its groups left)
        float* const mine = so + L::kMerge / 4;
        float2* const mine_ml = reinterpret_cast<float2*>(mine + ROWS * DP);
        for (int i = tid; i < rows * (DP / 4); i += THREADS) {
            const int row = i / (DP / 4), d = i % (DP / 4) * 4;
            float2 ml[4];
            float top = -INFINITY;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                ml[k] = sml[k * ROWS + row];
                top = fmaxf(top, ml[k].x);
            }
            const float ref = top == -INFINITY ? 0.0f : top;
            float sum = 0.0f;
            float4 y = make_float4(0, 0, 0, 0);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float f = ex2(ml[k].x - ref);
                const float4 v = *reinterpret_cast<const float4*>(so + (k * ROWS + row) * kP + d);
                sum += ml[k].y * f;
                y.x += v.x * f, y.y += v.y * f, y.z += v.z * f, y.w += v.w * f;
            }
            if (bad) sum = NAN;
            if constexpr (CLUSTER) {
                *reinterpret_cast<float4*>(mine + row * DP + d) = y;
                if (d == 0) mine_ml[row] = make_float2(top, sum);
            } else if (!whole) {
                *reinterpret_cast<float4*>(a.part_o + (part * ROWS + row) * DP + d) = y;
                if (d == 0) a.part_ml[part * ROWS + row] = make_float2(top, sum);
            } else if (d < c.dim) {
                const int R = mt * ROWS + row, j = R / a.group, g = R - j * a.group;
                const float f = vs / sum;
                T* dst = (T*)a.out +
                         (((long long)b * a.N + j) * a.q_heads + h * a.group + g) * c.dim + d;
                *reinterpret_cast<uint2*>(dst) =
                    make_uint2(pair<T>(y.x * f, y.y * f), pair<T>(y.z * f, y.w * f));
            }
        }
        if constexpr (CLUSTER) {
            // Every CTA adds up its share of the elements of all eight.
            cluster_sync();
            for (int i = cluster_rank() * THREADS + tid; i < rows * (DP / 4);
                 i += kCluster * THREADS) {
                const int row = i / (DP / 4), d = i % (DP / 4) * 4;
                if (d >= c.dim) continue;
                float2 ml[kCluster];
                float4 v[kCluster];
                float top = -INFINITY;
#pragma unroll
                for (int k = 0; k < kCluster; ++k) {
                    ml[k] = *cluster_at(mine_ml + row, k);
                    v[k] = *reinterpret_cast<const float4*>(cluster_at(mine + row * DP + d, k));
                    top = fmaxf(top, ml[k].x);
                }
                const float ref = top == -INFINITY ? 0.0f : top;
                float sum = 0.0f;
                float4 y = make_float4(0, 0, 0, 0);
#pragma unroll
                for (int k = 0; k < kCluster; ++k) {
                    const float f = ex2(ml[k].x - ref);
                    sum += ml[k].y * f;
                    y.x += v[k].x * f, y.y += v[k].y * f, y.z += v[k].z * f, y.w += v[k].w * f;
                }
                const int R = mt * ROWS + row, j = R / a.group, g = R - j * a.group;
                const float f = vs / sum;
                T* dst = (T*)a.out +
                         (((long long)b * a.N + j) * a.q_heads + h * a.group + g) * c.dim + d;
                *reinterpret_cast<uint2*>(dst) =
                    make_uint2(pair<T>(y.x * f, y.y * f), pair<T>(y.z * f, y.w * f));
            }
            cluster_sync();  // nobody leaves while its share is being read
            break;           // an item is all there is
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- many rows: tcgen05
//
// With more query rows per key head than mma.sync keeps up with, the products run on tcgen05.mma:
// 128 rows by 128 slots, scores, weights and outputs in tensor memory.  One CTA per SM; its warps
// have roles: one loads keys and one values (TMA, a box per page and panel of 64 elements, which
// swizzles rows of 128 bytes), two queries, one issues the products, 2 x 4 hold one query row per
// thread and turn scores into weights.  Two streams of scores alternate on the tensor
// pipe, so that one is multiplied while the other is exponentiated: two tiles of 128 rows over
// the same slots, or, when the rows fit one tile, every other 128 slots of it (joined at the
// end).  Work is cut into ranges and joined as for the split kernel, in units of 128 slots.
// Measured: 32 trees of 16 nodes, 128 rows per key head, 6000-12000 slots: 228 us, 5.5 TB/s (the
// chain scores - weights - product of a stream, 5000 cycles, hides all but a fifth of the memory's
// time); 8 trees of 65 nodes over 16000-33000 slots: 503 us, 867 TFLOP/s (the products: 128 x 128
// of two shared-memory operands takes all of that memory's bandwidth, 780 cycles where the tensor
// pipe alone would need 512); the same over float8: 264 us, 2.4 TB/s, and 643 us (making halves).

constexpr int kTcThreads = 512;
constexpr int kTcUnit = 128;  // slots
constexpr int kTcMaxCtas = 152;

constexpr int kBadFlags = 16;  // a power of two

template <int DP, int ROWS, bool F8> struct Tc {
    static constexpr int kTile = 128 * DP * 2;          // bytes of 128 keys, values or queries
    static constexpr int kQ = ROWS / 128 * kTile;
    // Stages: what fits beside the queries (the static part stays below 3 KiB), the odd one for
    // keys, which are wanted first.  float8: half as many stages of 16-bit operands, and what is
    // left for the bytes they are made of.
    static constexpr int kFit = (224 * 1024 - kQ) / kTile;
    static constexpr int kK = F8 ? (DP <= 64 ? 4 : 2) : kFit >= 12 ? 6 : (kFit + 1) / 2;
    static constexpr int kV = F8 ? (DP <= 64 ? 4 : 2) : kFit >= 12 ? 6 : kFit / 2;
    static constexpr int kRaw = 128 * DP;               // bytes of 128 float8 keys or values
    static constexpr int kRawFit = (224 * 1024 - kQ - (kK + kV) * kTile) / (2 * kRaw);
    static constexpr int kRaws = !F8 ? 0 : kRawFit > 4 ? 4 : kRawFit;  // of each
    static constexpr int kSmem = kQ + (kK + kV) * kTile + 2 * kRaws * kRaw;
    // A piece's bad page is flagged before the loads wait for a stage and looked at when its rows
    // are written.  With a tile per piece the loads of piece P have then met the products of piece
    // P - kRaws - kK - 1 (float8) or the scores of P - kK - 1, whose rows, or those of the piece
    // before, may still wait to be written: flags of so many pieces and one more are alive.
    static_assert(kK + kRaws + 3 <= kBadFlags, "flags of bad pages would be written over");
};

struct TcBars {
    uint64_t q_full, q_empty, epi_done, drain, v_land;
    uint64_t k_full[6], k_empty[6], v_full[6], v_empty[6];
    uint64_t s_full[2], p_full[2][2], pv_done[2];  // weights: a barrier per half of the slots
    uint64_t r_full[2][4], r_empty[2][4];  // float8 keys, values as they came
};

__device__ __forceinline__ uint32_t saddr(const void* p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void bar_init(uint64_t* bar, int count) {
    asm volatile("mbarrier.init.shared.b64 [%0], %1;" ::"r"(saddr(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared.b64 _, [%0];" ::"r"(saddr(bar)) : "memory");
}
// Arrives, expecting so many bytes of bulk copies besides.
__device__ __forceinline__ void bar_expect(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared.b64 _, [%0], %1;" ::"r"(saddr(bar)), "r"(bytes)
                 : "memory");
}
// One box of the cache: 64 elements from x of head h in slots from s on of page p.
__device__ __forceinline__ void tma_page(uint32_t dst, const CUtensorMap* map, int x, int h, int s,
                                         int p, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];"
        ::"r"(dst), "l"(map), "r"(x), "r"(h), "r"(s), "r"(p), "r"(saddr(bar)) : "memory");
}
constexpr uint32_t kGiveUp = 2000000000;  // two seconds
constexpr uint32_t kGap = 100000000;      // of them at most so much between two looks at the clock
__device__ __forceinline__ uint32_t nanoseconds() {
    uint32_t now;
    asm volatile("mov.u32 %0, %globaltimer_lo;" : "=r"(now));
    return now;
}
// What the waits of a CTA look at: whether one has given up, and how many products were issued.
struct Watch {
    int gave_up, issued;
};
// Waits for a phase of a barrier until two seconds have gone by without a product, or until another
// wait has given up; false when it gave up.  (Some wait for the end of a piece, which can take
// longer than any limit: a range of a context of 2^31 slots has 330000 tiles.)  A longer gap
// between two looks at the clock, as when the whole CTA was put aside for another process, counts
// as a tenth of a second: what was waited for then still has time to come.
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, volatile Watch* watch) {
    const uint32_t at = saddr(bar);
    uint32_t last = 0, waited = 0;
    int issued = -1;
    for (int i = 1;; ++i) {
        uint32_t done;
        asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared.b64 p, [%1], %2; "
                     "selp.u32 %0, 1, 0, p; }" : "=r"(done) : "r"(at), "r"(parity) : "memory");
        if (done) return true;
        if (i & 31) continue;
        const uint32_t now = nanoseconds();
        const int so_far = watch->issued;
        waited = so_far == issued ? waited + min(now - last, kGap) : 0;
        issued = so_far;
        last = now;
        if (watch->gave_up || waited > kGiveUp) break;
    }
    watch->gave_up = 1;
    return false;
}
// The same for a whole warp, with one answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile Watch* watch) {
    return __all_sync(~0u, bar_wait(bar, parity, watch));
}
__device__ __forceinline__ void named_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Shared-memory operand descriptor, 128-byte swizzle: rows of 128 bytes, 1024 bytes from one
// group of eight rows to the next; `panel`: bytes between panels of 64 elements, used where the
// operand's contiguous dimension is not the summed one (values: rows are slots).
__device__ __forceinline__ uint64_t operand(uint32_t at, uint32_t panel) {
    return (uint64_t)(at >> 4 & 0x3fff) | (uint64_t)(panel >> 4) << 16 |
           (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// Instruction descriptor: 128 x N, fp32 sums of bf16 or fp16 products; `rows`: the second
// operand's contiguous dimension is N.
template <typename T> __device__ __forceinline__ constexpr uint32_t product(int N, bool rows) {
    const uint32_t type = std::is_same<T, __half>::value ? 0u : 1u;
    return 1u << 4 | type << 7 | type << 10 | (rows ? 1u << 16 : 0u) | (uint32_t)(N >> 3) << 17 |
           (128u >> 4) << 24;
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t desc,
                                       bool add) {
    asm volatile("{ .reg .pred p; setp.ne.b32 p, %4, 0; "
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }"
                 ::"r"(d), "l"(a), "l"(b), "r"(desc), "r"((int)add) : "memory");
}
__device__ __forceinline__ void tc_mma_t(uint32_t d, uint32_t a, uint64_t b, uint32_t desc,
                                         bool add) {
    asm volatile("{ .reg .pred p; setp.ne.b32 p, %4, 0; "
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }"
                 ::"r"(d), "r"(a), "l"(b), "r"(desc), "r"((int)add) : "memory");
}
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                 ::"r"(saddr(bar)) : "memory");
}
// 32 columns of this thread's lane of tensor memory, as floats.
__device__ __forceinline__ void tc_ld32(float* r, uint32_t at) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
        "%28, %29, %30, %31}, [%32];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]),
          "=f"(r[6]), "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]),
          "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]), "=f"(r[17]),
          "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]),
          "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]),
          "=f"(r[30]), "=f"(r[31])
        : "r"(at) : "memory");
}
__device__ __forceinline__ void tc_st32(uint32_t at, const float* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, "
        "%10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, "
        "%27, %28, %29, %30, %31, %32};"
        ::"r"(at), "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]),
          "f"(r[7]), "f"(r[8]), "f"(r[9]), "f"(r[10]), "f"(r[11]), "f"(r[12]),
          "f"(r[13]), "f"(r[14]), "f"(r[15]), "f"(r[16]), "f"(r[17]), "f"(r[18]),
          "f"(r[19]), "f"(r[20]), "f"(r[21]), "f"(r[22]), "f"(r[23]), "f"(r[24]),
          "f"(r[25]), "f"(r[26]), "f"(r[27]), "f"(r[28]), "f"(r[29]), "f"(r[30]),
          "f"(r[31])
        : "memory");
}
__device__ __forceinline__ void tc_st32(uint32_t at, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
        ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
          "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
          "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
          "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
          "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]) : "memory");
}
__device__ __forceinline__ void tc_ld16(float* r, uint32_t at) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, "
        "%8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
          "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]),
          "=f"(r[14]), "=f"(r[15])
        : "r"(at) : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t at, const float* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, "
        "%9, %10, %11, %12, %13, %14, %15, %16};"
        ::"r"(at), "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]),
          "f"(r[7]), "f"(r[8]), "f"(r[9]), "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]),
          "f"(r[14]), "f"(r[15]) : "memory");
}
__device__ __forceinline__ float tc_ld1(uint32_t at) {
    float r;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];"
                 : "=f"(r) : "r"(at) : "memory");
    return r;
}
__device__ __forceinline__ void tc_wait_ld() {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

__device__ __forceinline__ bool elect_one() {
    uint32_t yes;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(yes));
    return yes != 0;
}

// float8 caches: the bytes land in stages of their own, and the four loading warps turn them into
// halves (exact) in the products' layout; a power of two is taken out of each bfloat16 query row
// so that it fits halves too, as in the split kernel.
template <typename T, typename CT, int DP, int ROWS>
__global__ void __launch_bounds__(kTcThreads, 1)
    kv_wide_kernel(const AttentionArgs a, const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap) {
    constexpr bool kF8 = sizeof(CT) == 1;
    using M = typename std::conditional<kF8, __half, T>::type;  // type of the products
    constexpr bool kFit = !kF8 || std::is_same<T, __half>::value;  // queries are of it already
    using L = Tc<DP, ROWS, kF8>;
    constexpr int SK = L::kK, SV = L::kV, CH = DP / 8;
    extern __shared__ __align__(1024) char smem_tc[];  // the swizzle counts from 1024
    __shared__ TcBars bars;
    __shared__ long long s_scan[kTcThreads / 32];
    __shared__ Start s_start;
    __shared__ Watch s_watch;
    __shared__ int s_bad_piece[kBadFlags], s_par[kMaxN];
    __shared__ uint64_t s_anc[kMaxN];
    __shared__ uint32_t s_tmem, s_wild[6][4];
    __shared__ float2 s_ml[128];
    __shared__ int8_t s_exp[2][ROWS];  // powers of two taken out of the queries, by piece parity
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const Cache& c = a.c;
    const uint32_t sq = saddr(smem_tc);  // queries, then stages of k, then of v
    const uint32_t sk = sq + L::kQ, sv = sk + SK * L::kTile, sr = sv + SV * L::kTile;

    if (tid == 0) {
        bar_init(&bars.q_full, 64);
        bar_init(&bars.q_empty, 1);
        bar_init(&bars.drain, 1);
        bar_init(&bars.epi_done, 256);
        bar_init(&bars.v_land, 1);
        constexpr int kFill = kF8 ? 128 : 1;
        for (int i = 0; i < SK; ++i) {
            bar_init(&bars.k_full[i], kFill);
            bar_init(&bars.k_empty[i], 1);
        }
        for (int i = 0; i < SV; ++i) {
            bar_init(&bars.v_full[i], kFill);
            bar_init(&bars.v_empty[i], 1);
        }
        for (int i = 0; i < 2 * L::kRaws; ++i) {
            bar_init(&bars.r_full[i & 1][i >> 1], 1);
            bar_init(&bars.r_empty[i & 1][i >> 1], 128);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(&bars.s_full[i], 1);
            bar_init(&bars.p_full[i][0], 128);
            bar_init(&bars.p_full[i][1], 128);
            bar_init(&bars.pv_done[i], 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        s_watch = Watch{0, 0};
    }
    if (tid < kBadFlags) s_bad_piece[tid] = -1;
    cudaGridDependencySynchronize();
    cudaTriggerProgrammaticLaunchCompletion();
    // (not before: a kernel that is still to end may have its own tensor memory to ask for)
    if (w == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(saddr(&s_tmem)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }

    tc_before();
    Walk walk = start_walk<kTcThreads>(a, ROWS, kTcUnit, s_scan, &s_start);
    tc_after();
    const uint32_t tmem = s_tmem;
    volatile Watch* watch = &s_watch;
    Piece p;

    if (kF8 && w >= 8 && w < 12) {
        // ------------------------------------------------ float8: bytes into halves
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        constexpr int kCh = DP / 16, R = L::kRaws > 0 ? L::kRaws : 1;  // 16-byte chunks of a row
        const int lt = tid - 256;
        int rs = 0, ds = 0;  // stages of bytes, of halves (keys and values have as many)
        uint32_t r_phase = 0, again = 1;
        bool ok = true;
        while (walk.next(a, ROWS, kTcUnit, &p)) {
            if (walk.sh.bad) continue;
            const int len = walk.sh.len, total = len + walk.sh.n;
            for (int t = p.t0; t < p.t1; ++t) {
#pragma unroll 1
                for (int kv = 0; kv < 2; ++kv) {
                    const bool tail = kv && (long long)(t + 1) * kTcUnit > len + 1;
                    ok = ok && warp_wait(&bars.r_full[kv][rs], r_phase, watch);
                    ok = ok &&
                         warp_wait(kv ? &bars.v_empty[ds] : &bars.k_empty[ds], again, watch);
                    if (tail) {
                        named_sync(2, 128);
                        if (lt < 4) s_wild[ds][lt] = 0;
                        named_sync(2, 128);
                    }
                    const uint32_t src = sr + (2 * rs + kv) * L::kRaw;
                    const uint32_t dst = (kv ? sv : sk) + ds * L::kTile;
                    auto read = [&](int i, uint32_t (&v)[4]) {
                        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                                     : "r"(src + i * 16) : "memory");
                    };
                    // Two 16-byte units per chunk; the lanes of the second panel write theirs in
                    // the other order, so that no two meet in a bank.
                    auto write = [&](int i, const uint32_t (&v)[4]) {
                        const int r = i / kCh, ch = i % kCh, flip = ch >> 2 & 1;
                        const uint32_t row = dst + (ch >> 2) * 16384 + r * 128;
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int u = k ^ flip;
                            uint32_t y[4];
                            widen(y[0], y[1], u ? v[2] : v[0]);
                            widen(y[2], y[3], u ? v[3] : v[1]);
                            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(
                                row + (((2 * ch + u & 7) ^ (r & 7)) << 4)),
                                "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]) : "memory");
                        }
                    };
                    if (!tail) {
#pragma unroll 1
                        for (int i = lt; i < 128 * kCh; i += 512) {
                            uint32_t v[4][4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) read(i + 128 * k, v[k]);
#pragma unroll
                            for (int k = 0; k < 4; ++k) write(i + 128 * k, v[k]);
                        }
                    } else {
                        // behind the last token: zeros; new tokens' NaN are zeroed here and added
                        // row by row
#pragma unroll 1
                        for (int i = lt; i < 128 * kCh; i += 128) {
                            uint32_t v[4];
                            read(i, v);
                            const int r = i / kCh;
                            const long long slot = (long long)t * kTcUnit + r;
                            bool wild = false;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                if (slot >= total) v[k] = 0;
#pragma unroll
                                for (int e = 0; e < 32; e += 8)
                                    if (slot > len && (v[k] >> e & 0x7f) == 0x7f) {
                                        wild = true;
                                        v[k] &= ~(0xffu << e);
                                    }
                            }
                            if (wild) atomicOr(&s_wild[ds][r >> 5], 1u << (r & 31));
                            write(i, v);
                        }
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    bar_arrive(&bars.r_empty[kv][rs]);
                    bar_arrive(kv ? &bars.v_full[ds] : &bars.k_full[ds]);
                }
                if (++rs == R) rs = 0, r_phase ^= 1;
                if (++ds == SK) ds = 0, again ^= 1;
            }
        }
    } else if (!kF8 && w >= 8 && w < 12) {
        // ------------------------------------------------ loads: a warp keys, a warp values
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        const bool vals = w > 8;  // warps 10 and 11 only help to look values through
        const int lt = tid - 288, stages = vals ? SV : SK;
        const CUtensorMap* const map = vals ? &vmap : &kmap;
        // A page is one box per panel (its first 128 slots where it is larger): this lane's page
        // of a tile.
        const int shift = min(c.page_shift, 7), boxes = kTcUnit >> shift;
        const uint32_t bytes = (128u << shift) * (DP / 64);  // per page
        int pieces = 0, st = 0;
        uint32_t again = 1, landed = 0;  // parities: the stage's last release; tails landed
        bool ok = true;  // once a wait gave up: no more copies, the barriers among the warps stay
        while (walk.next(a, ROWS, kTcUnit, &p)) {
            if (walk.sh.bad) continue;
            const int len = walk.sh.len, total = len + walk.sh.n;
            const int32_t* table = c.table + (long long)p.b * c.table_width;
            auto page_of = [&](int t) -> int {
                const long long s = (long long)t * kTcUnit + ((long long)lane << shift);
                return w < 10 && lane < boxes && t < p.t1 && s < total
                           ? __ldg(table + (s >> c.page_shift)) : -1;
            };
            int page = page_of(p.t0);
            for (int t = p.t0; t < p.t1; ++t) {
                const long long s = (long long)t * kTcUnit + ((long long)lane << shift);
                const uint32_t dst = (vals ? sv : sk) + st * L::kTile;
                const bool tail = vals && (long long)(t + 1) * kTcUnit > len + 1;
                uint64_t* const full = tail   ? &bars.v_land
                                       : vals ? &bars.v_full[st]
                                              : &bars.k_full[st];
                if (w < 10) {
                    const bool want = lane < boxes && s < total;
                    const bool good = want && (unsigned)page < (unsigned)c.num_pages;
                    if (want && !good) s_bad_piece[pieces % kBadFlags] = pieces;
                    const int pg = page;
                    page = page_of(t + 1);
                    ok = ok &&
                         warp_wait(vals ? &bars.v_empty[st] : &bars.k_empty[st], again, watch);
                    const uint32_t n = __popc(__ballot_sync(~0u, good));
                    if (ok) {
                        if (lane == 0) bar_expect(full, n * bytes);
                        __syncwarp();
                        if (good) {
                            const int slot = (int)(s & ((1 << c.page_shift) - 1));
#pragma unroll
                            for (int q = 0; q < DP / 64; ++q)
                                tma_page(dst + q * 16384 + (lane << shift) * 128, map, q * 64, p.h,
                                         slot, pg, full);
                        }
                    }
                }
                if (tail) {
                    // A masked entry may hold anything, but 0 times NaN is NaN: what lies behind
                    // the last token is zeroed here, and so are new tokens' values that are not
                    // finite; those are added row by row.
                    ok = ok && warp_wait(&bars.v_land, landed, watch);
                    landed ^= 1;
                    if (lt < 4) s_wild[st][lt] = 0;
                    named_sync(2, 96);
#pragma unroll 1
                    for (int r = lt; r < 128; r += 96) {  // a row per thread
                        const long long slot = (long long)t * kTcUnit + r;
                        if (slot <= len) continue;
                        constexpr uint32_t e = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
                        bool f = slot >= total;
#pragma unroll 4
                        for (int k = 0; k < CH; ++k) {
                            uint32_t v[4];
                            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                                         : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                                         : "r"(dst + (k >> 3) * 16384 + r * 128 +
                                               (((k & 7) ^ (r & 7)) << 4)) : "memory");
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                f |= (v[q] & e) == e || (v[q] >> 16 & e) == e;
                        }
                        if (!f) continue;
                        if (slot < total) atomicOr(&s_wild[st][r >> 5], 1u << (r & 31));
#pragma unroll 4
                        for (int k = 0; k < CH; ++k)
                            asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(
                                dst + (k >> 3) * 16384 + r * 128 + (((k & 7) ^ (r & 7)) << 4)),
                                "r"(0) : "memory");
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    named_sync(2, 96);
                    if (lt == 0) bar_arrive(&bars.v_full[st]);
                }
                if (++st == stages) st = 0, again ^= 1;
            }
            ++pieces;
        }
    } else if (w >= 12) {
        // ------------------------------------------------ products
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (kF8 && w == 15) {
            // float8: bytes of keys and values, a box per page
            const int shift = min(c.page_shift, 7), boxes = kTcUnit >> shift;
            constexpr int R = L::kRaws > 0 ? L::kRaws : 1;
            int pieces = 0, rs = 0;
            uint32_t again = 1;
            bool ok = true;
            while (ok && walk.next(a, ROWS, kTcUnit, &p)) {
                if (walk.sh.bad) continue;
                const int total = walk.sh.len + walk.sh.n;
                const int32_t* table = c.table + (long long)p.b * c.table_width;
                auto page_of = [&](int t) -> int {
                    const long long s = (long long)t * kTcUnit + ((long long)lane << shift);
                    return lane < boxes && t < p.t1 && s < total
                               ? __ldg(table + (s >> c.page_shift)) : -1;
                };
                int page = page_of(p.t0);
                for (int t = p.t0; ok && t < p.t1; ++t) {
                    const long long s = (long long)t * kTcUnit + ((long long)lane << shift);
                    const bool want = lane < boxes && s < total;
                    const bool good = want && (unsigned)page < (unsigned)c.num_pages;
                    if (want && !good) s_bad_piece[pieces % kBadFlags] = pieces;
                    const int pg = page, slot = (int)(s & ((1 << c.page_shift) - 1));
                    page = page_of(t + 1);
                    const uint32_t bytes =
                        __popc(__ballot_sync(~0u, good)) * ((uint32_t)DP << shift);
                    for (int kv = 0; ok && kv < 2; ++kv) {
                        ok = warp_wait(&bars.r_empty[kv][rs], again, watch);
                        if (!ok) break;
                        if (lane == 0) bar_expect(&bars.r_full[kv][rs], bytes);
                        __syncwarp();
                        if (good)
                            tma_page(sr + (2 * rs + kv) * L::kRaw + (lane << shift) * DP,
                                     kv ? &vmap : &kmap, 0, p.h, slot, pg, &bars.r_full[kv][rs]);
                        __syncwarp();
                    }
                    if (++rs == R) rs = 0, again ^= 1;
                }
                ++pieces;
            }
        }
        if (w == 13 || w == 14) {
            // queries: rows of the item, zeros past them
            const int lt = tid & 31 | (w - 13) << 5, dch = c.dim / 8;
            int pieces = 0;
            bool ok = true;
            while (ok && walk.next(a, ROWS, kTcUnit, &p)) {
                if (walk.sh.bad) continue;
                ok = warp_wait(&bars.q_empty, (pieces & 1) ^ 1, watch);
                auto query = [&](int row) {
                    const int R = p.mt * ROWS + (row < p.rows ? row : 0);
                    const int j = R / a.group, g = R - j * a.group;
                    return (const T*)a.q + p.b * a.qb + j * a.qt +
                           (long long)(p.h * a.group + g) * a.qh;
                };
                auto place = [&](int row, int ch) {
                    const int r = row & 127;
                    return sq + (row >> 7) * L::kTile + (ch >> 3) * 16384 + r * 128 +
                           (((ch & 7) ^ (r & 7)) << 4);
                };
                if constexpr (kFit) {
#pragma unroll 4
                    for (int i = lt; ok && i < ROWS * CH; i += 64) {
                        const int row = i / CH, ch = i % CH;
                        const bool take = row < p.rows && ch < dch;
                        cp_async16(place(row, ch), query(row) + (take ? ch * 8 : 0), take);
                    }
                    if (kF8)
                        for (int row = lt; row < ROWS; row += 64) s_exp[pieces & 1][row] = 0;
                    asm volatile("cp.async.wait_all;" ::: "memory");
                } else {
                    // eight lanes per row: its largest element becomes 2^8 .. 2^9; what then falls
                    // below the smallest half is 2^-33 of it
                    for (int row = lt >> 3; ok && row < ROWS; row += 8) {
                        const T* q = query(row);
                        Words<8> x[CH / 8];
                        float top = 0.0f;
#pragma unroll
                        for (int k = 0; k < CH / 8; ++k) {
                            const int ch = k * 8 + (lane & 7);
                            x[k] = Words<8>{};
                            if (row < p.rows && ch < dch) x[k] = get<8>(q + ch * 8);
                            float f[8];
                            widen_to<T, 8>(f, x[k]);
#pragma unroll
                            for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(f[e]));
                        }
                        for (int k = 4; k; k >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, k));
                        const int e2 = row_power(top);
                        const float down = exp2f((float)-e2);
                        if ((lane & 7) == 0) s_exp[pieces & 1][row] = (int8_t)e2;
#pragma unroll
                        for (int k = 0; k < CH / 8; ++k) {
                            float f[8];
                            widen_to<T, 8>(f, x[k]);
                            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(
                                place(row, k * 8 + (lane & 7))),
                                "r"(pair<__half>(f[0] * down, f[1] * down)),
                                "r"(pair<__half>(f[2] * down, f[3] * down)),
                                "r"(pair<__half>(f[4] * down, f[5] * down)),
                                "r"(pair<__half>(f[6] * down, f[7] * down)) : "memory");
                        }
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                bar_arrive(&bars.q_full);
                ++pieces;
            }
        }
        if (w == 12 && elect_one()) {
            const uint32_t pv = product<M>(c.dim, true);  // the elements that heads have
            constexpr uint32_t kPanel = DP > 64 ? 16384 : 1024;  // one panel: not used
            // scores times the sign of the scales: the largest is then the one to look for
            constexpr uint32_t kNegate = 1u << 13;
            uint32_t qk = product<M>(128, false);
            const uint64_t qd = operand(sq, 16384), kd = operand(sk, 16384);
            const uint64_t vd = operand(sv, kPanel);
            constexpr int kStep = L::kTile >> 4;  // a tile further in a descriptor
            int ks = 0, vs = 0;  // stages and parities of the next tiles of keys and of values
            uint32_t k_phase = 0, v_phase = 0, pieces = 0, p_phase = 0;
            int issued = 0;
            bool ok = true;
            while (ok && walk.next(a, ROWS, kTcUnit, &p)) {
                if (walk.sh.bad) continue;
                const bool two = p.rows > 128;
                const int nt = p.t1 - p.t0, jobs = two ? 2 * nt : nt;
                const bool negate = (a.scale < 0.0f) != (kF8 && c.k_scale[p.h] < 0.0f);
                qk = negate ? qk | kNegate : qk & ~kNegate;
                ok = bar_wait(&bars.q_full, pieces & 1, watch);
                // Job i belongs to stream i & 1.  Its scores take the place of the weights of job
                // i - 2, whose product comes before them; products of one thread run in order.
                // Each stream's product and next scores are issued together, so that the streams
                // take turns.
                auto scores = [&](int i) {
                    const int st = i & 1;
                    if (!two || st == 0) ok = ok && bar_wait(&bars.k_full[ks], k_phase, watch);
                    if (!ok) return;
                    const uint64_t qa = qd + (two ? st * kStep : 0), ka = kd + ks * kStep;
#pragma unroll
                    for (int k = 0; k < DP / 16; ++k) {
                        if (k * 16 >= c.dim) break;
                        // in 16 bytes: a panel, 16 elements of a row
                        const uint64_t at = (k >> 2) * (16384 >> 4) + (k & 3) * 2;
                        tc_mma(tmem + st * 128, qa + at, ka + at, qk, k > 0);
                    }
                    tc_commit(&bars.s_full[st]);
                    if (!two || st == 1) {
                        tc_commit(&bars.k_empty[ks]);
                        if (++ks == SK) ks = 0, k_phase ^= 1;
                    }
                    if (i == jobs - 1) tc_commit(&bars.q_empty);
                };
                if (ok) scores(0);
                if (ok && jobs > 1) scores(1);
                for (int i = 0; ok && i < jobs; ++i) {
                    const int st = i & 1;
                    if (!two || st == 0) ok = bar_wait(&bars.v_full[vs], v_phase, watch);
                    const uint64_t va = vd + vs * kStep;
                    const uint32_t pd = tmem + st * 128, od = tmem + 256 + st * DP;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        ok = ok && bar_wait(&bars.p_full[st][half], p_phase >> st & 1, watch);
                        if (!ok) break;
                        tc_after();
#pragma unroll
                        for (int k = 4 * half; k < 4 * half + 4; ++k)
                            tc_mma_t(od, pd + (k >> 1) * 32 + (k & 1) * 8, va + k * 128, pv, true);
                    }
                    p_phase ^= 1u << st;
                    if (!ok) break;
                    tc_commit(&bars.pv_done[st]);
                    watch->issued = ++issued;
                    if (!two || st == 1) {
                        tc_commit(&bars.v_empty[vs]);
                        if (++vs == SV) vs = 0, v_phase ^= 1;
                    }
                    if (i + 2 < jobs) scores(i + 2);
                }
                ++pieces;
            }
            if (!ok) {  // products in flight end before the tensor memory goes back
                volatile Watch alone = {0, 0};
                tc_commit(&bars.drain);
                bar_wait(&bars.drain, 0, &alone);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------ weights: a row per thread
        asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        const int st = w >> 2, r = tid & 127;
        const uint32_t mine = tmem + ((uint32_t)(w & 3) * 32 << 16);
        const uint32_t sc = mine + st * 128, oc = mine + 256 + st * DP;
        uint32_t s_phase = 0, pv = 0;  // phases of the scores; products waited for
        long long tiles = 0;
        int pieces = 0, anc_of = -1;
        bool tree_bad = false, ok = true;  // a wait that gave up skips the rest, not the barriers
        while (walk.next(a, ROWS, kTcUnit, &p)) {
            const Share& sh = walk.sh;
            const bool two = p.rows > 128;
            const int row = two ? st * 128 + r : r, R = p.mt * ROWS + row;
            const int j = min(R / a.group, sh.n - 1), g = R - R / a.group * a.group;
            const bool live = row < p.rows;
            if (tid == 0) tell_ends(a, p, sh.tiles);
            T* out = (T*)a.out +
                     (((long long)p.b * a.N + j) * a.q_heads + p.h * a.group + g) * c.dim;
            if (sh.bad) {
                if (live && (two || st == 0))
                    for (int d = 0; d < c.dim; ++d) out[d] = Conv<T>::from(NAN);
                __syncwarp();
                continue;
            }
            const int len = sh.len, nt = p.t1 - p.t0, jobs = two ? 2 * nt : nt;
            if ((long long)p.t1 * kTcUnit > len && anc_of != p.b) {
                named_sync(1, 256);
                int f = 0;
                if (a.parents && tid < sh.n) {
                    const int q = a.parents[(long long)p.b * a.N + tid];
                    s_par[tid] = q;
                    f = tid > 0 && (q < 0 || q >= tid);
                }
                // any bad parent: every thread learns it from the barrier's reduction
                asm volatile("{ .reg .pred p, q; setp.ne.b32 p, %1, 0; "
                             "barrier.cta.red.or.pred q, 1, 256, p; selp.s32 %0, 1, 0, q; }"
                             : "=r"(f) : "r"(f) : "memory");
                if (tid < sh.n) {
                    uint64_t m = 0;
                    if (!a.parents)
                        m = tid == 64 ? ~0ull : (1ull << tid) - 1;
                    else if (!f)
                        for (int i = tid; i > 0; i = s_par[i]) m |= 1ull << (i - 1);
                    s_anc[tid] = m;
                }
                named_sync(1, 256);
                anc_of = p.b;
                tree_bad = f;
                if (f && tid == 0) mark(a.status, p.b, SV_DEV_BAD_TREE);
            }
            const bool nan_rows = tree_bad && anc_of == p.b;
            const uint64_t anc = anc_of == p.b ? s_anc[j] : 0;
            // from a score to an exponent of two; the products carry the sign
            const float unit0 = fabsf(a.scale) * 1.4426950408889634f;
            const float ks_h = kF8 ? fabsf(c.k_scale[p.h]) : 1.0f;
            float unit = unit0 * ks_h;
            const bool busy = (two ? st * 128 : 0) + (w & 3) * 32 < p.rows;  // rows in this warp
            float l = 0.0f, ref = -INFINITY;
            int done = 0;  // jobs of this stream
            // the outputs of the piece before have been read; this one's start at zero
            ok = ok && warp_wait(&bars.epi_done, (pieces & 1) ^ 1, watch);
            tc_after();
            {
                float zero[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) zero[e] = 0.0f;
#pragma unroll
                for (int k = 0; k < DP; k += 32) tc_st32(oc + k, zero);
                tc_wait_st();
            }
            for (int i = st; ok && i < jobs; i += 2, ++done) {
                const int t = p.t0 + (two ? i >> 1 : i);
                ok = warp_wait(&bars.s_full[st], s_phase, watch);
                s_phase ^= 1;
                if (!ok) break;
                tc_after();
                if (!kFit && done == 0)
                    unit = unit0 * exp2f((float)s_exp[pieces & 1][row]) * ks_h;
                if (!busy) {  // rows that nothing comes of: any weights will do
                    tc_before();
                    bar_arrive(&bars.p_full[st][0]);
                    bar_arrive(&bars.p_full[st][1]);
                    continue;
                }
                const bool tail = (long long)(t + 1) * kTcUnit > len + 1;
                uint32_t see[4];  // of the tile's slots, those that this row sees
                if (tail) {
                    const int rel = t * kTcUnit - len;  // slot 0 of the tile among the new tokens
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int at = rel + 32 * k - 1;  // bit of anc for the word's first slot
                        see[k] = at >= 64    ? 0u
                                 : at >= 0   ? (uint32_t)(anc >> at)
                                 : at > -32  ? (uint32_t)(anc << -at) | ((1u << -at) - 1)
                                             : ~0u;
                    }
                }
                float x[128];
#pragma unroll
                for (int k = 0; k < 128; k += 32) tc_ld32(x + k, sc + k);
                tc_wait_ld();
                if (tail) {
#pragma unroll
                    for (int e = 0; e < 128; ++e)
                        if (!(see[e >> 5] >> (e & 31) & 1)) x[e] = -INFINITY;
                }
                float m[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                for (int e = 4; e < 124; e += 8)
#pragma unroll
                    for (int k = 0; k < 4; ++k) m[k] = fmaxf(fmaxf(m[k], x[e + k]), x[e + k + 4]);
#pragma unroll
                for (int k = 0; k < 4; ++k) m[k] = fmaxf(m[k], x[124 + k]);
                const float top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
                const float mx = top == -INFINITY ? -INFINITY : top * unit;
                // The reference follows the maximum only when that has grown by 2^8.
                const bool grow = mx > ref + 8.0f;
                bool waited = false;  // for the product before this one
                if (__any_sync(~0u, grow)) {
                    const float f = grow ? ex2(ref - mx) : 1.0f;
                    if (grow) ref = mx;
                    l *= f;
                    if (done > 0) {
                        ok = warp_wait(&bars.pv_done[st], (pv + done - 1) & 1, watch);
                        waited = true;
                        tc_after();
#pragma unroll 1
                        for (int k = 0; k < DP; k += 16) {
                            float o[16];
                            tc_ld16(o, oc + k);
                            tc_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] *= f;
                            tc_st16(oc + k, o);
                        }
                        tc_wait_st();
                    }
                }
                const float less = ref == -INFINITY ? 0.0f : ref;
                if (tail) {
                    const long long tile = tiles + (two ? i >> 1 : i);
                    const int vs = (int)(tile % SV);
                    ok = ok && warp_wait(&bars.v_full[vs], (uint32_t)(tile / SV & 1), watch);
#pragma unroll 1
                    for (int sl = 0; ok && sl < 128; ++sl) {
                        if (!(s_wild[vs][sl >> 5] >> (sl & 31) & 1)) continue;
                        if (done > 0 && !waited) {
                            ok = warp_wait(&bars.pv_done[st], (pv + done - 1) & 1, watch);
                            waited = true;
                            tc_after();
                        }
                        const int n = t * kTcUnit + sl - len;  // the new token, >= 1
                        const float y = tc_ld1(sc + sl);
                        tc_wait_ld();
                        const bool mine_too = sees(anc, n);
                        const float pw = mine_too ? ex2(y * unit - less) : 0.0f;
                        const long long at = slot_offset(c, p.b, len + n);
                        const CT* v = (const CT*)(c.v + (at < 0 ? 0 : at) + p.h * c.head_stride);
#pragma unroll 1
                        for (int k = 0; k < c.dim; k += 16) {
                            float o[16];
                            tc_ld16(o, oc + k);
                            tc_wait_ld();
                            if (mine_too && at >= 0) {
#pragma unroll
                                for (int e = 0; e < 16; ++e) {
                                    const float y = Conv<CT>::to(v[k + e]);
                                    // (of float8 rows only what is not finite was zeroed)
                                    if (!kF8 || y != y) o[e] += pw * y;
                                }
                            }
                            __syncwarp();
                            tc_st16(oc + k, o);
                            tc_wait_st();
                        }
                    }
                }
                // Weights take the place of scores, in pairs: 16 columns of each 32.  They are
                // rounded to the products' 16-bit type once, which leaves about as much of an
                // error as rounding the result; low halves for them too (a second product) took
                // a tenth longer on trees of 16 nodes (263 against 239 us).
                float2 sum[2] = {{0, 0}, {0, 0}};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float y[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float2 v = fma2(make_float2(x[32 * k + 2 * e], x[32 * k + 2 * e + 1]),
                                        make_float2(unit, unit), make_float2(-less, -less));
                        v.x = ex2(v.x);
                        v.y = ex2(v.y);
                        if (tail) {
                            if (!(see[k] >> (2 * e) & 1)) v.x = 0.0f;
                            if (!(see[k] >> (2 * e + 1) & 1)) v.y = 0.0f;
                        }
                        sum[e & 1] = add2(sum[e & 1], v);
                        y[e] = __uint_as_float(pair<M>(v.x, v.y));
                    }
                    tc_st16(sc + 32 * k, y);
                    if (k & 1) {  // half of the slots: their product may begin
                        tc_wait_st();
                        tc_before();
                        bar_arrive(&bars.p_full[st][k >> 1]);
                    }
                }
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            }
            // the stream's last product
            if (ok && done > 0) ok = warp_wait(&bars.pv_done[st], (pv + done - 1) & 1, watch);
            pv += done;
            tc_after();
            const bool whole = p.t0 == 0 && p.t1 == sh.tiles;
            float f0 = 1.0f, f1 = 0.0f;  // shares of the two streams where they are joined
            if (!two) {
                if (st == 1) s_ml[r] = make_float2(ref, l);
                tc_before();
                named_sync(1, 256);
                tc_after();
                if (st == 0 && jobs > 1) {
                    const float2 o = s_ml[r];
                    const float top = fmaxf(ref, o.x), less = top == -INFINITY ? 0.0f : top;
                    f0 = ex2(ref - less);
                    f1 = ex2(o.x - less);
                    l = l * f0 + o.y * f1;
                    ref = top;
                }
            }
            // Whatever wait of the CTA gave up (the other stream's, a load's), the rows may be made
            // of anything: its flag was set before what came here.
            const bool late = !ok || watch->gave_up;
            const bool bad_page = s_bad_piece[pieces % kBadFlags] == pieces;
            if (late && r == 0) mark(a.status, p.b, SV_DEV_TIMEOUT);
            if (bad_page && !nan_rows && tid == 0) mark(a.status, p.b, SV_DEV_BAD_PAGE);
            if (two || st == 0) {
                if (nan_rows || bad_page || late) l = NAN;
                const long long part = 2 * (long long)blockIdx.x + (p.t0 == 0 ? 1 : 0);
                const float inv = (kF8 ? c.v_scale[p.h] : 1.0f) / l;
#pragma unroll 1
                for (int k = 0; k < DP; k += 32) {
                    float o[32];
                    tc_ld32(o, oc + k);
                    tc_wait_ld();
                    if (!two) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] *= f0;
                        if (jobs > 1) {
                            float y[32];
                            tc_ld32(y, oc + DP + k);
                            tc_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] += y[e] * f1;
                        }
                    }
                    if (live && !whole) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4*>(
                                a.part_o + ((part * (DP / 4) + (k + e) / 4) * ROWS + row) * 4) =
                                make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    } else if (live) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            if (k + e >= c.dim) continue;
                            uint32_t y[4];
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                y[q] = pair<T>(o[e + 2 * q] * inv, o[e + 2 * q + 1] * inv);
                            *reinterpret_cast<uint4*>(out + k + e) =
                                make_uint4(y[0], y[1], y[2], y[3]);
                        }
                    }
                    __syncwarp();
                }
                if (live && !whole) a.part_ml[part * ROWS + row] = make_float2(ref, l);
            }
            tc_before();
            bar_arrive(&bars.epi_done);
            tiles += nt;
            ++pieces;
        }
    }
    if (watch->gave_up) {  // loads that nobody waited for land within a millisecond
        const uint32_t since = nanoseconds();
        while (nanoseconds() - since < 1000000) __nanosleep(1000);
    }
    tc_before();
    __syncthreads();
    tc_after();
    if (w == 12)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
}

// Adds up the pieces of the items that more than one range holds, at most one per range that
// starts one: sum over pieces of 2^(m - max) (o, l), then o / l.  A CTA of four warps per four
// rows of an item (a warp each), or per row (the warps share its pieces) where the host expects
// many pieces per item.
template <typename T, int DP>
__global__ void __launch_bounds__(128) kv_join_kernel(const AttentionArgs a, int rows, int warps) {
    __shared__ float4 s_o[4][DP / 4];
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const Cache& c = a.c;
    cudaGridDependencySynchronize();
    const int item = a.started[blockIdx.x];
    if (item < 0) return;
    const int mt = item % a.mts, h = item / a.mts % c.heads, b = item / a.mts / c.heads;
    const int c0 = blockIdx.x, c1 = a.ended[item];
    const Share sh = share_of(a, b, rows, kUnit);
    const int row = warps == 1 ? blockIdx.y * 4 + w : blockIdx.y;
    const int live = min(rows, sh.n * a.group - mt * rows);
    const bool mine = row < live;
    if (warps == 4 && !mine) return;
    // piece i of c0 .. c1: the first starts the item (slot 1 of its CTA), the others continue it
    auto at = [&](int i) { return (long long)(2 * i + (i == c0 ? 1 : 0)) * rows + row; };
    float top = -INFINITY, L = 0.0f;
    float4 y = make_float4(0, 0, 0, 0);
    if (mine) {
        for (int i = c0 + lane; i <= c1; i += 32) top = fmaxf(top, a.part_ml[at(i)].x);
        for (int k = 16; k; k >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, k));
        const float ref = top == -INFINITY ? 0.0f : top;
        for (int i = c0 + lane; i <= c1; i += 32) {
            const float2 ml = a.part_ml[at(i)];
            L += ml.y * ex2(ml.x - ref);
        }
        for (int k = 16; k; k >>= 1) L += __shfl_xor_sync(~0u, L, k);
        if (lane < DP / 4) {
            const int first = c0 + (warps == 4 ? w : 0);
#pragma unroll 8
            for (int i = first; i <= c1; i += warps) {
                const float f = ex2(a.part_ml[at(i)].x - ref);
                const float4 v = *reinterpret_cast<const float4*>(a.part_o + at(i) * DP + lane * 4);
                y.x += v.x * f, y.y += v.y * f, y.z += v.z * f, y.w += v.w * f;
            }
        }
    }
    if (warps == 4) {
        if (lane < DP / 4) s_o[w][lane] = y;
        __syncthreads();
        if (w) return;
        if (lane < DP / 4)
            for (int k = 1; k < 4; ++k) {
                const float4 v = s_o[k][lane];
                y.x += v.x, y.y += v.y, y.z += v.z, y.w += v.w;
            }
    }
    if (!mine || lane * 4 >= c.dim) return;
    const int R = mt * rows + row, j = R / a.group, g = R - j * a.group;
    const float f = (c.v_scale ? c.v_scale[h] : 1.0f) / L;
    T* dst =
        (T*)a.out + (((long long)b * a.N + j) * a.q_heads + h * a.group + g) * c.dim + lane * 4;
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(pair<T>(y.x * f, y.y * f), pair<T>(y.z * f, y.w * f));
}

// The same for pieces of the wide kernel: a warp takes 32 rows by four elements, so that what it
// reads lies together, as it was written; the four warps of a CTA neighbouring elements, or (many
// pieces) a quarter of the pieces each.
template <typename T, int DP>
__global__ void __launch_bounds__(128) kv_wide_join_kernel(const AttentionArgs a, int rows,
                                                           int warps) {
    __shared__ float s_y[3][32][5];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const Cache& c = a.c;
    cudaGridDependencySynchronize();
    const int item = a.started[blockIdx.x];
    if (item < 0) return;
    const int mt = item % a.mts, h = item / a.mts % c.heads, b = item / a.mts / c.heads;
    const int c0 = blockIdx.x, c1 = a.ended[item];
    const Share sh = share_of(a, b, rows, kTcUnit);
    const int cols = DP / 4 / (warps == 4 ? 1 : 4);  // blocks of four elements, or of sixteen
    const int row = blockIdx.y / cols * 32 + lane;
    const int d4 = warps == 4 ? blockIdx.y % cols : blockIdx.y % cols * 4 + w;
    const bool live = row < min(rows, sh.n * a.group - mt * rows) && d4 * 4 < c.dim;
    if (warps == 1 && !live) return;
    auto at = [&](int i) { return (long long)(2 * i + (i == c0 ? 1 : 0)); };
    float top = -INFINITY, L = 0.0f;
    float4 y = make_float4(0, 0, 0, 0);
    if (live) {
#pragma unroll 8
        for (int i = c0; i <= c1; ++i) top = fmaxf(top, a.part_ml[at(i) * rows + row].x);
        const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll 8
        for (int i = c0 + (warps == 4 ? w : 0); i <= c1; i += warps) {
            const float2 ml = a.part_ml[at(i) * rows + row];
            const float f = ex2(ml.x - ref);
            const float4 v = *reinterpret_cast<const float4*>(
                a.part_o + ((at(i) * (DP / 4) + d4) * rows + row) * 4);
            L += ml.y * f;
            y.x += v.x * f, y.y += v.y * f, y.z += v.z * f, y.w += v.w * f;
        }
    }
    if (warps == 4) {
        if (w) {
            float* to = s_y[w - 1][lane];
            to[0] = y.x, to[1] = y.y, to[2] = y.z, to[3] = y.w, to[4] = L;
        }
        __syncthreads();
        if (w || !live) return;
        for (int k = 0; k < 3; ++k) {
            const float* of = s_y[k][lane];
            y.x += of[0], y.y += of[1], y.z += of[2], y.w += of[3], L += of[4];
        }
    }
    const int R = mt * rows + row, j = R / a.group, g = R - j * a.group;
    const float f = (c.v_scale ? c.v_scale[h] : 1.0f) / L;
    T* dst = (T*)a.out + (((long long)b * a.N + j) * a.q_heads + h * a.group + g) * c.dim + d4 * 4;
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(pair<T>(y.x * f, y.y * f), pair<T>(y.z * f, y.w * f));
}

// ---------------------------------------------------------------- commit

struct CommitArgs {
    Cache c;
    long long layer_stride;  // bytes
    const int32_t* kv_len;
    const int32_t* out_nodes;
    const int32_t* num_accepted;
    int32_t* kv_len_out;
    uint32_t* status;
    int N, units;  // 16-byte units of one slot's entry, all heads
    int head_units;
    int planes, run;  // layers' keys and values; how many of them a CTA takes
};

constexpr int kCommitThreads = 128;
constexpr int kCommitBatch = 8;
constexpr int kCommitResident = 8;  // CTAs per SM

// One CTA per sequence and run of planes (a layer's keys or values).  Accepted nodes increase, so
// those that stay where they are (node i + 1 in place i) come first and the rest moves.  Each
// thread owns one 16-byte column of the entries; for each plane it moves the column of all nodes
// in order, eight moves at a time (of several planes, where one has fewer): the sources of a batch
// are read before any of its targets is written, and since a_i >= i increases, no target is the
// source of a later batch.  Bound by the latency of reads of scattered entries (a thread waits for
// its eight; a third of the warps that fit are there, DRAM 36 % busy on half the sequences), for a
// few rows by the chain node - page - entry: every moved entry is read once and written once (256
// trees of 65 nodes, 16 float8 layers: 33 us, 4.8 TB/s; one layer of one tree 3.1 us).
__global__ void __launch_bounds__(kCommitThreads, kCommitResident)
    kv_commit_kernel(const CommitArgs a) {
    __shared__ long long s_src[kMaxN], s_dst[kMaxN];
    const int b = blockIdx.z, tid = threadIdx.x;
    const Cache& c = a.c;
    const int n = a.num_accepted[b], len = a.kv_len[b];
    // (asked for before n is known: the row has N nodes)
    const int32_t* nodes = a.out_nodes + (long long)b * a.N;
    const int node = a.out_nodes && tid < a.N ? nodes[tid] : 0;
    const int before = a.out_nodes && tid > 0 && tid < a.N ? nodes[tid - 1] : 0;
    const bool first = blockIdx.x == 0 && blockIdx.y == 0 && tid == 0;
    const long long cap = (long long)c.table_width << c.page_shift;
    uint32_t bad = 0;
    int stay = 0;
    if (n < -1 || n >= a.N || len < 0 || (long long)len + n + 1 > cap) {
        bad = SV_DEV_BAD_LENGTH;
    } else if (n > 0 && a.out_nodes) {
        int f = 0;
        const bool stays = tid < n && node == tid + 1;
        if (tid < n) {
            if (node <= before || node >= a.N) {
                f = SV_DEV_BAD_TREE;
            } else if ((long long)len + node >= cap) {
                f = SV_DEV_BAD_LENGTH;
            } else if (!stays) {
                s_src[tid] = slot_offset(c, b, len + node);
                s_dst[tid] = slot_offset(c, b, len + tid + 1);
                if (s_src[tid] < 0 || s_dst[tid] < 0) f = SV_DEV_BAD_PAGE;
            }
        }
        stay = __syncthreads_count(stays);
        if (__syncthreads_or(f))
            bad = __syncthreads_or(f & SV_DEV_BAD_TREE)     ? SV_DEV_BAD_TREE
                  : __syncthreads_or(f & SV_DEV_BAD_LENGTH) ? SV_DEV_BAD_LENGTH
                                                            : SV_DEV_BAD_PAGE;
    }
    if (first) {
        if (bad) mark(a.status, b, bad);
        a.kv_len_out[b] = bad ? len : len + n + 1;
    }
    if (bad || n <= 0 || !a.out_nodes) return;
    // entries shorter than the block: planes side by side
    const int side = a.units < kCommitThreads ? kCommitThreads / a.units : 1;
    const int lane = a.units < kCommitThreads ? tid / a.units : 0;
    const int u = blockIdx.x * kCommitThreads + tid - lane * a.units;
    if (u >= a.units || lane >= side) return;
    const int h = u / a.head_units;
    const long long column = h * c.head_stride + (u - h * a.head_units) * 16;
    const int p0 = blockIdx.y * a.run, p1 = min(a.planes, p0 + a.run);
    int plane = p0 + lane, move = stay;
    while (plane < p1 && stay < n) {
        uint4 x[kCommitBatch];
        char* to[kCommitBatch];
#pragma unroll
        for (int i = 0; i < kCommitBatch; ++i) {
            to[i] = nullptr;
            if (plane >= p1) continue;
            char* base = (plane & 1 ? c.v : c.k) + (plane >> 1) * a.layer_stride + column;
            x[i] = *reinterpret_cast<const uint4*>(base + s_src[move]);
            to[i] = base + s_dst[move];
            if (++move == n) move = stay, plane += side;
        }
#pragma unroll
        for (int i = 0; i < kCommitBatch; ++i)
            if (to[i]) *reinterpret_cast<uint4*>(to[i]) = x[i];
    }
}

// ---------------------------------------------------------------- host

static int elem_bytes(sv_dtype t) { return t == SV_E4M3 ? 1 : 2; }
static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Calls f with the types and sizes of the split kernel that these sizes take: 16 query rows
// of a key head per CTA, or 32 where there are more (one CTA then reads each key once for all).
template <bool CLUSTER, typename F>
static auto with_split(sv_dtype dtype, sv_dtype cache, int dim, int rows, F f) {
    auto sized = [&](auto t, auto ct) {
        using T = decltype(t);
        using CT = decltype(ct);
        if (dim <= 64)
            return rows <= 16 ? f(kv_split_kernel<T, CT, 64, 1, CLUSTER>, kv_join_kernel<T, 64>,
                                  Split<CT, 64, 1>::kSmem)
                              : f(kv_split_kernel<T, CT, 64, 2, CLUSTER>, kv_join_kernel<T, 64>,
                                  Split<CT, 64, 2>::kSmem);
        return rows <= 16 ? f(kv_split_kernel<T, CT, 128, 1, CLUSTER>, kv_join_kernel<T, 128>,
                              Split<CT, 128, 1>::kSmem)
                          : f(kv_split_kernel<T, CT, 128, 2, CLUSTER>, kv_join_kernel<T, 128>,
                              Split<CT, 128, 2>::kSmem);
    };
    if (dtype == SV_BF16)
        return cache == SV_E4M3 ? sized(__nv_bfloat16(), __nv_fp8_e4m3())
                                : sized(__nv_bfloat16(), __nv_bfloat16());
    return cache == SV_E4M3 ? sized(__half(), __nv_fp8_e4m3()) : sized(__half(), __half());
}

// The same for the wide kernel: tiles of 128 rows, or of two times 128.
template <typename F>
static auto with_wide(sv_dtype dtype, sv_dtype cache, int dim, int rows, F f) {
    auto sized = [&](auto t, auto ct) {
        using T = decltype(t);
        using CT = decltype(ct);
        constexpr bool F8 = sizeof(CT) == 1;
        if (dim <= 64)
            return rows <= 128 ? f(kv_wide_kernel<T, CT, 64, 128>, kv_wide_join_kernel<T, 64>,
                                   Tc<64, 128, F8>::kSmem)
                               : f(kv_wide_kernel<T, CT, 64, 256>, kv_wide_join_kernel<T, 64>,
                                   Tc<64, 256, F8>::kSmem);
        return rows <= 128 ? f(kv_wide_kernel<T, CT, 128, 128>, kv_wide_join_kernel<T, 128>,
                               Tc<128, 128, F8>::kSmem)
                           : f(kv_wide_kernel<T, CT, 128, 256>, kv_wide_join_kernel<T, 128>,
                               Tc<128, 256, F8>::kSmem);
    };
    if (dtype == SV_BF16)
        return cache == SV_E4M3 ? sized(__nv_bfloat16(), __nv_fp8_e4m3())
                                : sized(__nv_bfloat16(), __nv_bfloat16());
    return cache == SV_E4M3 ? sized(__half(), __nv_fp8_e4m3()) : sized(__half(), __half());
}

// Whether a call takes a cluster per item: when all its clusters are resident at once and a CTA's
// share of the longest context that the table can hold is at most 16 units (1024 slots).
static bool small_call(int B, int heads, int rows, int slots, int sms) {
    const long long items = (long long)B * heads * ((rows + (rows <= 16 ? 15 : 31)) /
                                                    (rows <= 16 ? 16 : 32));
    return items * kCluster <= 2 * sms && slots <= kCluster * 16 * kUnit;
}

// A cache tensor as the TMA sees it: element, head, slot, page.  False where it does not take the
// strides (2^40 bytes and more).
static bool cache_map(CUtensorMap* map, void* base, const sv_kv_cache* c) {
    static PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                             &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            f = nullptr;
        return (PFN_cuTensorMapEncodeTiled_v12000)f;
    }();
    if (!encode) return false;
    const int e = elem_bytes(c->dtype);
    const cuuint64_t dims[4] = {(cuuint64_t)c->dim, (cuuint64_t)c->heads, (cuuint64_t)c->page_size,
                                (cuuint64_t)c->num_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)c->head_stride * e, (cuuint64_t)c->slot_stride * e,
                                   (cuuint64_t)c->page_stride * e};
    // rows of 128 bytes, swizzled, for the products; float8 rows whole, as they are
    const bool f8 = c->dtype == SV_E4M3;
    const cuuint32_t box[4] = {f8 && c->dim > 64 ? 128u : 64u, 1,
                               (cuuint32_t)(c->page_size < 128 ? c->page_size : 128), 1};
    const cuuint32_t step[4] = {1, 1, 1, 1};
    return encode(map,
                  f8                    ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                  : c->dtype == SV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                        : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                  4, base, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  f8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Shared memory of the many-row kernels.  *can: false where a compiler gave them other registers
// than their roles share out (256 threads of 184, 256 of 72: those of a launch with 128 each; with
// fewer the larger share would be waited for).
static bool wide_setup(bool* can) {
    bool ok = true;
    *can = true;
    for (int i = 0; i < 16 && ok; ++i) {
        const sv_dtype t = i & 1 ? SV_F16 : SV_BF16;
        ok = with_wide(t, i & 2 ? SV_E4M3 : t, i & 4 ? 128 : 64, i & 8 ? 256 : 128,
                       [&](auto k, auto, int smem) {
            cudaFuncAttributes f;
            if (cudaFuncGetAttributes(&f, k) != cudaSuccess) return false;
            *can = *can && f.numRegs == 128;
            return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) ==
                   cudaSuccess;
        });
    }
    return ok;
}
// The same of the others.
static bool split_setup() {
    auto set = [](auto k, auto, int smem) {
        return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) ==
               cudaSuccess;
    };
    bool ok = true;
    for (sv_dtype t : {SV_BF16, SV_F16})
        for (sv_dtype ct : {t, SV_E4M3})
            for (int dim : {64, 128})
                for (int rows : {16, 32})
                    ok = ok && with_split<false>(t, ct, dim, rows, set) &&
                         with_split<true>(t, ct, dim, rows, set);
    return ok;
}

// The current device's SM count, if it is one that these kernels run on.  wide (attention): whether
// the many-row kernels can be launched; the split kernel takes any number of rows.
static sv_status device_ok(int* sms, bool* wide = nullptr) {
    struct Known {
        int sms;        // 0 unknown, -1 another device
        int attention;  // 0 unknown, 1 without the many-row kernels, 2 with them
    };
    static std::mutex mu;
    static Known known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SV_ERR_CUDA;
    if (dev < 0 || dev >= 64) return SV_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lk(mu);
    Known& k = known[dev];
    if (!k.sms) {
        int major = 0, minor = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
            return SV_ERR_CUDA;
        int n = -1;
        if (major == 10 && minor == 3 &&
            cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return SV_ERR_CUDA;
        k.sms = n;
    }
    if (k.sms < 0) return SV_ERR_UNSUPPORTED;
    *sms = k.sms;
    if (!wide) return SV_OK;
    if (!k.attention) {
        bool can;
        if (!split_setup() || !wide_setup(&can)) return SV_ERR_CUDA;
        k.attention = can ? 2 : 1;
    }
    *wide = k.attention == 2;
    return SV_OK;
}

// The workspace: where items are cut (tiles of at least 16 rows, of 32 where there are more), then
// two pieces of a row tile per CTA.
struct AttentionWs { size_t part_o, part_ml, bytes; };
static AttentionWs attention_ws(int B, int heads, int rows, int dim) {
    const size_t dp = dim <= 64 ? 64 : 128, items = (size_t)B * heads * ((rows + 31) / 32);
    const size_t split = (size_t)2 * kMaxCtas * (rows <= 16 ? 16 : 32);
    const size_t wide = rows <= 32 ? 0 : (size_t)2 * kTcMaxCtas * (rows <= 128 ? 128 : 256);
    const size_t held = split > wide ? split : wide;
    AttentionWs l;
    l.part_o = ((items + kMaxCtas) * sizeof(int) + 255) / 256 * 256;
    l.part_ml = l.part_o + held * dp * 4;
    l.bytes = l.part_ml + held * 8;
    return l;
}

// scales: the call needs the scales of a float8 cache.
static sv_status check_cache(const sv_kv_cache* c, bool scales, int B, Cache* out) {
    if (!c || !c->k || !c->v || (B > 0 && !c->table)) return SV_ERR_INVALID_ARG;
    if (!aligned16(c->k) || !aligned16(c->v) || !aligned16(c->table)) return SV_ERR_INVALID_ARG;
    if (c->dtype != SV_BF16 && c->dtype != SV_F16 && c->dtype != SV_E4M3) return SV_ERR_INVALID_ARG;
    const bool scaled = c->dtype == SV_E4M3;
    if (scales && (scaled != (c->k_scale != nullptr) || scaled != (c->v_scale != nullptr)))
        return SV_ERR_INVALID_ARG;
    if (c->num_pages < 1 || c->page_size < 1 || c->table_width < 1 || c->heads < 1 || c->dim < 1)
        return SV_ERR_INVALID_ARG;
    if ((c->page_size & (c->page_size - 1)) || c->dim % 16 || c->dim > kMaxDim ||
        c->heads > kMaxQHeads || (int64_t)c->table_width * c->page_size >= (1ll << 31))
        return SV_ERR_UNSUPPORTED;
    const int e = elem_bytes(c->dtype);
    const int64_t s[3] = {c->page_stride, c->slot_stride, c->head_stride};
    for (int64_t x : s)
        if (x < c->dim || x > (1ll << 40) || x * e % 16) return SV_ERR_INVALID_ARG;
    *out = Cache{(char*)c->k, (char*)c->v, c->table, c->k_scale, c->v_scale,
                 c->page_stride * e, c->slot_stride * e, c->head_stride * e,
                 c->num_pages, __builtin_ctz(c->page_size), c->table_width, c->heads, c->dim};
    return SV_OK;
}

static bool overlap(const int32_t* a, const int32_t* b, int n) { return a < b + n && b < a + n; }

static bool strides_ok(const sv_strides* s) {
    if (!s) return false;
    const int64_t x[3] = {s->batch, s->token, s->head};
    for (int64_t v : x)
        if (v < 0 || v > (1ll << 40) || v % 8) return false;
    return true;
}

// Sizes and the arguments that append and attention share.
static sv_status check_tokens(const sv_kv_cache* c, sv_dtype dtype, const int32_t* kv_len,
                              const int32_t* num_new, const int32_t* parents,
                              const uint32_t* status, int B, int N, int q_heads) {
    if (dtype != SV_BF16 && dtype != SV_F16) return SV_ERR_INVALID_ARG;
    if (c->dtype != dtype && c->dtype != SV_E4M3) return SV_ERR_INVALID_ARG;
    if (B < 0 || N < 1) return SV_ERR_INVALID_ARG;
    if (q_heads < 1 || q_heads % c->heads) return SV_ERR_INVALID_ARG;
    if (N > kMaxN || B > kMaxB || q_heads > kMaxQHeads) return SV_ERR_UNSUPPORTED;
    if (B > 0 && !kv_len) return SV_ERR_INVALID_ARG;
    if (!aligned16(kv_len) || !aligned16(num_new) || !aligned16(parents) || !aligned16(status))
        return SV_ERR_INVALID_ARG;
    return SV_OK;
}

template <typename T, typename CT>
static void launch_append(AppendArgs& a, int B, int sms, cudaStream_t s) {
    // whole 16-byte accesses when the rotated part allows it
    const int V = a.rot % 16 == 0 ? 8 : a.rot % 8 == 0 ? 4 : 1;
    const int units = a.c.dim / (2 * V), heads = (a.q ? a.q_heads : 0) + 2 * a.c.heads;
    // A head per thread where that makes a small block, else two (and more passes past that).
    const int want = heads * units <= 256 ? heads : (heads + kAppendHeads - 1) / kAppendHeads;
    const int side_by_side = want < kAppendThreads / units ? want : kAppendThreads / units;
    // Runs of tokens once there are more of them than CTAs resident twice over: a run pays its
    // chain of lengths, pages and angles once (16640 tokens of 80 heads: a token per CTA 179 us,
    // four 120 us); fewer tokens are spread over the SMs.
    const long long tokens = (long long)a.N * B / (6ll * sms);
    a.run = tokens < 1 ? 1 : tokens > kAppendTokens ? kAppendTokens : (int)tokens;
    const dim3 grid((a.N + a.run - 1) / a.run, B), block(units, side_by_side);
    auto go = [&](auto kernel) { kernel<<<grid, block, 0, s>>>(a); };
    if (V == 8)
        a.interleaved ? go(kv_append_kernel<T, CT, 8, true>)
                      : go(kv_append_kernel<T, CT, 8, false>);
    else if (V == 4)
        a.interleaved ? go(kv_append_kernel<T, CT, 4, true>)
                      : go(kv_append_kernel<T, CT, 4, false>);
    else
        a.interleaved ? go(kv_append_kernel<T, CT, 1, true>)
                      : go(kv_append_kernel<T, CT, 1, false>);
}

static sv_status launched() { return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA; }

}  // namespace svkv

using namespace svkv;

extern "C" {

sv_status spec_kv_rope_turns(int rot_dim, double base, double factor, double original_length,
                             double low, double high, uint64_t* turns) {
    if (!turns || rot_dim < 2 || rot_dim % 2 || rot_dim > kMaxDim) return SV_ERR_INVALID_ARG;
    if (!(base > 1.0) || !std::isfinite(base) || !(factor >= 1.0) || !std::isfinite(factor) ||
        !std::isfinite(original_length) || !std::isfinite(low) || !std::isfinite(high))
        return SV_ERR_INVALID_ARG;
    if (original_length > 0 && !(low < high)) return SV_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586476925286766559;
    for (int i = 0; i < rot_dim / 2; ++i) {
        const double rate = std::pow(base, -2.0 * i / rot_dim) / two_pi;  // turns per position
        double keep = 0.0;
        if (original_length > 0) {
            keep = (original_length * rate - low) / (high - low);
            keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
        }
        const double r = keep * rate + (1.0 - keep) * rate / factor;  // below 1/2pi
        turns[i] = (uint64_t)std::llround(std::ldexp(r, 62)) << 2;
    }
    return SV_OK;
}

sv_status spec_kv_append(const sv_kv_cache* cache, const sv_rope* rope, const void* q,
                         const sv_strides* q_strides, const void* k, const void* v,
                         const sv_strides* kv_strides, sv_dtype dtype, const int32_t* kv_len,
                         const int32_t* num_new, const int32_t* tree_parents, int B, int N,
                         int q_heads, void* q_out, uint32_t* status, cudaStream_t stream) {
    AppendArgs a = {};
    sv_status st = check_cache(cache, true, B, &a.c);
    if (st != SV_OK) return st;
    if (!q) q_heads = cache->heads;
    st = check_tokens(cache, dtype, kv_len, num_new, tree_parents, status, B, N, q_heads);
    if (st != SV_OK) return st;
    if (!strides_ok(kv_strides) || (q && !strides_ok(q_strides))) return SV_ERR_INVALID_ARG;
    if (B > 0 && (!k || !v || (q && !q_out))) return SV_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || (q && !aligned16(q_out)))
        return SV_ERR_INVALID_ARG;
    if (q && q == q_out &&
        (q_strides->head != cache->dim || q_strides->token != (int64_t)q_heads * cache->dim ||
         q_strides->batch != (int64_t)N * q_heads * cache->dim))
        return SV_ERR_INVALID_ARG;  // in place only where both have the same layout
    if (rope) {
        if (!rope->turns || !aligned16(rope->turns) || rope->rot_dim < 2 || rope->rot_dim % 2 ||
            rope->rot_dim > cache->dim || !std::isfinite(rope->magnitude) ||
            (rope->interleaved != 0 && rope->interleaved != 1))
            return SV_ERR_INVALID_ARG;
        a.turns = rope->turns;
        a.rot = rope->rot_dim;
        a.interleaved = rope->interleaved;
        a.magnitude = rope->magnitude;
    }
    if (B == 0) return SV_OK;
    int sms;
    if ((st = device_ok(&sms)) != SV_OK) return st;
    a.q = (const char*)q;
    a.k = (const char*)k;
    a.v = (const char*)v;
    a.q_out = (char*)q_out;
    if (q) a.qb = q_strides->batch, a.qt = q_strides->token, a.qh = q_strides->head;
    a.kb = kv_strides->batch, a.kt = kv_strides->token, a.kh = kv_strides->head;
    a.kv_len = kv_len;
    a.num_new = num_new;
    a.parents = tree_parents;
    a.status = status;
    a.N = N;
    a.q_heads = q_heads;
    if (dtype == SV_BF16) {
        if (cache->dtype == SV_E4M3)
            launch_append<__nv_bfloat16, __nv_fp8_e4m3>(a, B, sms, stream);
        else
            launch_append<__nv_bfloat16, __nv_bfloat16>(a, B, sms, stream);
    } else {
        if (cache->dtype == SV_E4M3)
            launch_append<__half, __nv_fp8_e4m3>(a, B, sms, stream);
        else
            launch_append<__half, __half>(a, B, sms, stream);
    }
    return launched();
}

size_t spec_kv_attention_workspace_size(int B, int N, int q_heads, int heads, int dim) {
    if (B < 0 || B > kMaxB || N < 1 || N > kMaxN || heads < 1 || q_heads < 1 || q_heads % heads ||
        q_heads > kMaxQHeads || dim < 16 || dim > kMaxDim || dim % 16)
        return 0;
    return attention_ws(B, heads, N * (q_heads / heads), dim).bytes;
}

sv_status spec_kv_attention(const sv_kv_cache* cache, const void* q, const sv_strides* q_strides,
                            sv_dtype dtype, const int32_t* kv_len, const int32_t* num_new,
                            const int32_t* tree_parents, float scale, int B, int N, int q_heads,
                            void* out, void* ws, size_t ws_bytes, uint32_t* status,
                            cudaStream_t stream) {
    AttentionArgs a = {};
    sv_status st = check_cache(cache, true, B, &a.c);
    if (st != SV_OK) return st;
    st = check_tokens(cache, dtype, kv_len, num_new, tree_parents, status, B, N, q_heads);
    if (st != SV_OK) return st;
    if (!strides_ok(q_strides) || !std::isfinite(scale)) return SV_ERR_INVALID_ARG;
    if (B > 0 && (!q || !out)) return SV_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(out)) return SV_ERR_INVALID_ARG;
    if (!ws) return SV_ERR_WORKSPACE;
    if (!aligned16(ws)) return SV_ERR_INVALID_ARG;
    if (ws_bytes < spec_kv_attention_workspace_size(B, N, q_heads, cache->heads, cache->dim))
        return SV_ERR_WORKSPACE;
    if (B == 0) return SV_OK;
    int sms;
    bool wide;
    if ((st = device_ok(&sms, &wide)) != SV_OK) return st;
    a.q = (const char*)q;
    a.out = (char*)out;
    a.qb = q_strides->batch, a.qt = q_strides->token, a.qh = q_strides->head;
    a.kv_len = kv_len;
    a.num_new = num_new;
    a.parents = tree_parents;
    a.status = status;
    a.scale = scale;
    a.N = N;
    a.q_heads = q_heads;
    a.group = q_heads / cache->heads;
    a.B = B;
    // Few items over short contexts: a cluster each, in one launch.  Else few rows: mma.sync,
    // which then waits for memory only; more: tcgen05, where a page fills whole groups of eight
    // rows of the swizzle.
    const int rows = N * a.group;
    const bool cluster =
        small_call(B, cache->heads, rows, cache->table_width * cache->page_size, sms);
    // Float8 over short contexts stays with mma.sync up to 64 rows: pieces of one or two units, and
    // no halves to make (100 sequences, 8 key heads of 128, 64 rows each over at most 128 slots 70
    // against 118 us, 2000 slots 235 against 252, 3000 slots 313 against 295).
    const int slots = cache->table_width * cache->page_size;
    const int few = cache->dtype == SV_E4M3 && slots <= 2048 ? 64 : 32;
    CUtensorMap kmap, vmap;
    wide = wide && !cluster && rows > few && cache->page_size >= 8 &&
           cache_map(&kmap, cache->k, cache) && cache_map(&vmap, cache->v, cache);
    const int tile = wide ? (rows <= 128 ? 128 : 256) : rows <= 16 ? 16 : 32;
    const int unit = wide ? kTcUnit : kUnit;
    const int mts = (rows + tile - 1) / tile;
    if ((long double)B * cache->heads * mts *
            ((double)cache->table_width * cache->page_size / unit + 1) >= (long double)(1ll << 50))
        return SV_ERR_UNSUPPORTED;
    if ((long long)B * cache->heads * mts >= (1ll << 31)) return SV_ERR_UNSUPPORTED;  // grid size
    const int most = wide ? kTcMaxCtas : kMaxCtas, fit = wide ? sms : 2 * sms;
    a.ctas = fit < most ? fit : most;
    const AttentionWs l = attention_ws(B, cache->heads, rows, cache->dim);
    a.mts = mts;
    a.started = (int*)ws;
    a.ended = a.started + kMaxCtas;
    a.part_o = (float*)((char*)ws + l.part_o);
    a.part_ml = (float2*)((char*)ws + l.part_ml);
    // Pieces per item, if all sequences were alike: with many, the warps of a CTA share a row.
    const int warps = a.ctas >= 8 * (long long)B * cache->heads * mts ? 4 : 1;
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = kCluster;
    attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
    auto launch = [&](auto kernel, auto join, int smem) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(cluster ? B * cache->heads * mts * kCluster : a.ctas);
        cfg.blockDim = dim3(wide ? kTcThreads : kSplitThreads * tile / 16);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        cfg.attrs = attrs;
        cfg.numAttrs = cluster ? 2 : 1;
        cudaError_t r;
        if constexpr (std::is_same<decltype(kernel), void (*)(const AttentionArgs)>::value ||
                      std::is_same<decltype(kernel), void (*)(AttentionArgs)>::value)
            r = cudaLaunchKernelEx(&cfg, kernel, a);
        else
            r = cudaLaunchKernelEx(&cfg, kernel, a, kmap, vmap);
        if (r != cudaSuccess || cluster) return r;
        cfg.numAttrs = 1;
        cfg.blockDim = dim3(128);
        cfg.dynamicSmemBytes = 0;
        const int parts = wide ? tile / 32 * (cache->dim <= 64 ? 16 : 32) : tile;
        cfg.gridDim = dim3(a.ctas, warps == 4 ? parts : parts / 4);
        return cudaLaunchKernelEx(&cfg, join, a, tile, warps);
    };
    const cudaError_t e = wide ? with_wide(dtype, cache->dtype, cache->dim, rows, launch)
                    : cluster ? with_split<true>(dtype, cache->dtype, cache->dim, rows, launch)
                              : with_split<false>(dtype, cache->dtype, cache->dim, rows, launch);
    return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

sv_status spec_kv_commit(const sv_kv_cache* cache, int layers, int64_t layer_stride,
                         const int32_t* kv_len, const int32_t* out_nodes,
                         const int32_t* num_accepted, int B, int N, int32_t* kv_len_out,
                         uint32_t* status, cudaStream_t stream) {
    CommitArgs a = {};
    sv_status st = check_cache(cache, false, B, &a.c);
    if (st != SV_OK) return st;
    if (layers < 1 || B < 0 || N < 1) return SV_ERR_INVALID_ARG;
    const int e = elem_bytes(cache->dtype);
    if (layers > 1 && (layer_stride < cache->dim || layer_stride > (1ll << 40) ||
                       layer_stride * e % 16))
        return SV_ERR_INVALID_ARG;
    if (N > kMaxN || B > kMaxB || layers > 32767) return SV_ERR_UNSUPPORTED;
    if (B > 0 && (!kv_len || !num_accepted || !kv_len_out)) return SV_ERR_INVALID_ARG;
    if (!aligned16(kv_len) || !aligned16(out_nodes) || !aligned16(num_accepted) ||
        !aligned16(kv_len_out) || !aligned16(status))
        return SV_ERR_INVALID_ARG;
    if (B == 0) return SV_OK;
    // a CTA may still read a sequence's length or count when another writes its new length
    if (overlap(kv_len_out, kv_len, B) || overlap(kv_len_out, num_accepted, B))
        return SV_ERR_INVALID_ARG;
    int sms;
    if ((st = device_ok(&sms)) != SV_OK) return st;
    a.layer_stride = layers > 1 ? layer_stride * e : 0;
    a.kv_len = kv_len;
    a.out_nodes = out_nodes;
    a.num_accepted = num_accepted;
    a.kv_len_out = kv_len_out;
    a.status = status;
    a.N = N;
    a.head_units = cache->dim * e / 16;
    a.units = cache->heads * a.head_units;
    // As many CTAs as are resident at once: a CTA's chain node - page is paid once per run.
    const long long ctas = (a.units + kCommitThreads - 1) / kCommitThreads;
    a.planes = 2 * layers;
    a.run = (int)(((long long)a.planes * ctas * B + kCommitResident * sms - 1) /
                  (kCommitResident * sms));
    const int side = a.units < kCommitThreads ? kCommitThreads / a.units : 1;
    a.run = a.run < side ? side : a.run;
    a.run = a.run > a.planes ? a.planes : a.run;
    const dim3 grid((unsigned)ctas, (a.planes + a.run - 1) / a.run, B);
    kv_commit_kernel<<<grid, kCommitThreads, 0, stream>>>(a);
    return launched();
}

}  // extern "C"
