// The paged key-value cache of a speculative round: append with rotation,
// attention of the drafted tokens, commit of the accepted ones
// (include/specverify_kv.h).

#include "specverify_kv.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cmath>
#include <cstdint>
#include <mutex>

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
    // round to nearest, saturating at +-448 (infinities too); NaN stays NaN
    static __device__ __nv_fp8_e4m3 from(float x) { return __nv_fp8_e4m3(x); }
};

// V elements of type T moved as one access (2 V or V bytes, aligned to them).
template <typename T, int V> struct alignas(sizeof(T) * V) Vec { T x[V]; };

// ---------------------------------------------------------------- sequences

// Tokens of sequence b, or -1 for a bad length.
__device__ __forceinline__ int new_tokens(const int32_t* kv_len, const int32_t* num_new, int b,
                                          int N, const Cache& c, int* len) {
    const int n = num_new ? num_new[b] : N;
    const int l = kv_len[b];
    *len = l;
    const long long cap = (long long)c.table_width << c.page_shift;
    if (n < 0 || n > N || l < 0 || (long long)l + n > cap) return -1;
    return n;
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
    int N, q_heads;
};

constexpr int kAppendThreads = 256;

// One CTA per new token: it forms the token's cosines and sines once, in shared
// memory, and turns every head with them.  The angle is position * rate modulo
// one turn in 64-bit integers (exact), so far positions lose nothing; its top 32
// bits become the argument of sincospi.  V pairs of a head per step: 2 V elements
// of 2 bytes read and written in 16-byte accesses when V = 8.  Bound by memory:
// each query, key and value is read once and written once.
template <typename T, typename CT, int V>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendArgs a) {
    __shared__ float2 s_cs[kMaxDim / 2];
    __shared__ int s_par[kMaxN];
    const int b = blockIdx.y, j = blockIdx.x, tid = threadIdx.x;
    const Cache& c = a.c;
    int len;
    const int n = new_tokens(a.kv_len, a.num_new, b, a.N, c, &len);
    if (n < 0) {
        if (j == 0 && tid == 0) mark(a.status, b, SV_DEV_BAD_LENGTH);
        return;
    }
    if (j >= n) return;
    int depth = j;
    if (a.parents) {
        int bad = 0;
        for (int i = tid; i < n; i += kAppendThreads) {
            const int p = a.parents[(long long)b * a.N + i];
            s_par[i] = p;
            bad |= i > 0 && (p < 0 || p >= i);
        }
        if (__syncthreads_or(bad)) {
            if (j == 0 && tid == 0) mark(a.status, b, SV_DEV_BAD_TREE);
            return;
        }
        depth = 0;
        for (int i = j; i > 0; i = s_par[i]) ++depth;
    }
    const int half = a.rot / 2;
    const uint64_t pos = (uint64_t)len + depth;
    for (int i = tid; i < half; i += kAppendThreads) {
        const int32_t t = (int32_t)((pos * a.turns[i]) >> 32);
        float s, co;
        sincospif((float)t * 4.656612873077393e-10f, &s, &co);  // 2^-31: half turns
        s_cs[i] = make_float2(co * a.magnitude, s * a.magnitude);
    }
    const long long place = slot_offset(c, b, len + j);
    if (place < 0 && tid == 0) mark(a.status, b, SV_DEV_BAD_PAGE);
    __syncthreads();

    // Units of a head: rot/2/V rotated ones (2 V elements each), then the rest in
    // steps of V; of a value head: dim/V steps.
    const int D = c.dim, turn_units = half / V, units = turn_units + (D - a.rot) / V;
    const int qn = a.q ? a.q_heads : 0;
    const int heads = qn + c.heads;
    using VT = Vec<T, V>;
    using VC = Vec<CT, V>;
    for (int u = tid; u < heads * units; u += kAppendThreads) {
        const int h = u / units, w = u - h * units;
        const bool is_q = h < qn;
        const T* src = is_q ? (const T*)a.q + b * a.qb + j * a.qt + h * a.qh
                            : (const T*)a.k + b * a.kb + j * a.kt + (h - qn) * a.kh;
        int e0, e1;
        float r0[V], r1[V];
        const bool turns = w < turn_units;
        if (turns) {
            e0 = a.interleaved ? 2 * w * V : w * V;
            e1 = a.interleaved ? e0 + V : e0 + half;
        } else {
            e0 = a.rot + (w - turn_units) * V;
            e1 = e0;
        }
        const VT x0 = *reinterpret_cast<const VT*>(src + e0);
#pragma unroll
        for (int i = 0; i < V; ++i) r0[i] = Conv<T>::to(x0.x[i]);
        if (turns) {
            const VT x1 = *reinterpret_cast<const VT*>(src + e1);
#pragma unroll
            for (int i = 0; i < V; ++i) r1[i] = Conv<T>::to(x1.x[i]);
            if (a.interleaved) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float2 cs = s_cs[w * V + i];
                    // pair i of the unit: elements 2i and 2i + 1 of its 2 V
                    float& x = 2 * i < V ? r0[2 * i < V ? 2 * i : 0] : r1[2 * i < V ? 0 : 2 * i - V];
                    float& y = 2 * i + 1 < V ? r0[2 * i + 1 < V ? 2 * i + 1 : 0]
                                             : r1[2 * i + 1 < V ? 0 : 2 * i + 1 - V];
                    const float p = x * cs.x - y * cs.y;
                    y = y * cs.x + x * cs.y;
                    x = p;
                }
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float2 cs = s_cs[w * V + i];
                    const float p = r0[i] * cs.x - r1[i] * cs.y;
                    r1[i] = r1[i] * cs.x + r0[i] * cs.y;
                    r0[i] = p;
                }
            }
        }
        if (is_q) {
            T* dst = (T*)a.q_out + (((long long)b * a.N + j) * a.q_heads + h) * D;
            VT y;
#pragma unroll
            for (int i = 0; i < V; ++i) y.x[i] = Conv<T>::from(r0[i]);
            *reinterpret_cast<VT*>(dst + e0) = y;
            if (turns) {
#pragma unroll
                for (int i = 0; i < V; ++i) y.x[i] = Conv<T>::from(r1[i]);
                *reinterpret_cast<VT*>(dst + e1) = y;
            }
        } else if (place >= 0) {
            CT* dst = (CT*)(c.k + place + (h - qn) * c.head_stride);
            const float ks = c.k_scale ? c.k_scale[h - qn] : 1.0f;
            VC y;
#pragma unroll
            for (int i = 0; i < V; ++i)
                y.x[i] = Conv<CT>::from(c.k_scale ? __fdiv_rn(r0[i], ks) : r0[i]);
            *reinterpret_cast<VC*>(dst + e0) = y;
            if (turns) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    y.x[i] = Conv<CT>::from(c.k_scale ? __fdiv_rn(r1[i], ks) : r1[i]);
                *reinterpret_cast<VC*>(dst + e1) = y;
            }
        }
    }
    if (place < 0) return;
    constexpr int W = 8;  // dim is a multiple of 16
    for (int u = tid; u < c.heads * (D / W); u += kAppendThreads) {
        const int h = u / (D / W), e = (u - h * (D / W)) * W;
        const T* src = (const T*)a.v + b * a.kb + j * a.kt + h * a.kh + e;
        const Vec<T, W> x = *reinterpret_cast<const Vec<T, W>*>(src);
        CT* dst = (CT*)(c.v + place + h * c.head_stride) + e;
        if constexpr (sizeof(CT) == sizeof(T)) {
            *reinterpret_cast<Vec<T, W>*>(dst) = x;
        } else {
            const float vs = c.v_scale[h];
            Vec<CT, W> y;
#pragma unroll
            for (int i = 0; i < W; ++i) y.x[i] = Conv<CT>::from(__fdiv_rn(Conv<T>::to(x.x[i]), vs));
            *reinterpret_cast<Vec<CT, W>*>(dst) = y;
        }
    }
}

// ---------------------------------------------------------------- attention

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
    int N, q_heads, group;
};

constexpr int kSimpleThreads = 128;

// One CTA per query row, a warp per cached position in turn, each warp with its
// own running maximum, sum and output; the four warps are joined at the end.
template <typename T, typename CT>
__global__ void __launch_bounds__(kSimpleThreads) kv_attention_kernel(const AttentionArgs a) {
    __shared__ int s_par[kMaxN];
    __shared__ float s_m[4], s_l[4], s_o[4][kMaxDim];
    const int b = blockIdx.z, j = blockIdx.y, h = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const Cache& c = a.c;
    int len;
    const int n = new_tokens(a.kv_len, a.num_new, b, a.N, c, &len);
    if (n >= 0 && j >= n) return;
    uint32_t bad = n < 0 ? SV_DEV_BAD_LENGTH : 0;
    T* out = (T*)a.out + (((long long)b * a.N + j) * a.q_heads + h) * c.dim;
    int bad_tree = 0;
    if (!bad && a.parents) {
        for (int i = tid; i < n; i += kSimpleThreads) {
            const int p = a.parents[(long long)b * a.N + i];
            s_par[i] = p;
            bad_tree |= i > 0 && (p < 0 || p >= i);
        }
        if (__syncthreads_or(bad_tree)) bad = SV_DEV_BAD_TREE;
    }
    if (!bad) {
        int bp = 0;
        for (int p = tid; p < (len + n + (1 << c.page_shift) - 1) >> c.page_shift; p += kSimpleThreads)
            bp |= (unsigned)c.table[(long long)b * c.table_width + p] >= (unsigned)c.num_pages;
        if (__syncthreads_or(bp)) bad = SV_DEV_BAD_PAGE;
    }
    if (bad) {
        if (tid == 0 && j == 0 && h == 0) mark(a.status, b, bad);
        for (int d = tid; d < c.dim; d += kSimpleThreads) out[d] = Conv<T>::from(NAN);
        return;
    }
    uint64_t seen = 0;  // bit i - 1: node i is node j or an ancestor of it
    if (!a.parents)
        seen = j == 64 ? ~0ull : (1ull << j) - 1;
    else
        for (int i = j; i > 0; i = s_par[i]) seen |= 1ull << (i - 1);
    const int kh = h / a.group, D = c.dim, per = 4;  // lane: elements 4 lane ..
    const T* q = (const T*)a.q + b * a.qb + j * a.qt + h * a.qh;
    float qf[4], o[4] = {0, 0, 0, 0};
    const float ks = (c.k_scale ? c.k_scale[kh] : 1.0f) * a.scale;
    for (int i = 0; i < per; ++i) qf[i] = lane * 4 + i < D ? Conv<T>::to(q[lane * 4 + i]) : 0.0f;
    float m = -INFINITY, l = 0;
    for (int s = w; s < len + n; s += 4) {
        if (s > len && !(seen >> (s - len - 1) & 1)) continue;
        const long long at = slot_offset(c, b, s) + kh * c.head_stride;
        const CT* kp = (const CT*)(c.k + at);
        const CT* vp = (const CT*)(c.v + at);
        float x = 0, vv[4];
        for (int i = 0; i < per; ++i) {
            const int d = lane * 4 + i;
            x += d < D ? qf[i] * Conv<CT>::to(kp[d]) : 0.0f;
            vv[i] = d < D ? Conv<CT>::to(vp[d]) : 0.0f;
        }
        for (int k = 16; k; k >>= 1) x += __shfl_xor_sync(~0u, x, k);
        x *= ks;
        const float mn = fmaxf(m, x);
        const float base = mn == -INFINITY ? 0.0f : mn;
        const float f = __expf(m - base), p = __expf(x - base);
        l = l * f + p;
        for (int i = 0; i < per; ++i) o[i] = o[i] * f + p * vv[i];
        m = mn;
    }
    if (lane == 0) s_m[w] = m, s_l[w] = l;
    for (int i = 0; i < per; ++i) s_o[w][lane * 4 + i] = o[i];
    __syncthreads();
    float M = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
    if (M == -INFINITY) M = 0;
    const float vs = c.v_scale ? c.v_scale[kh] : 1.0f;
    for (int d = tid; d < D; d += kSimpleThreads) {
        float L = 0, O = 0;
        for (int i = 0; i < 4; ++i) {
            const float f = s_l[i] == 0 && s_m[i] == -INFINITY ? 0.0f : __expf(s_m[i] - M);
            L += s_l[i] * f;
            O += f == 0 && s_l[i] == 0 ? 0.0f : s_o[i][d] * f;
        }
        out[d] = Conv<T>::from(O / L * vs);
    }
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
};

constexpr int kCommitThreads = 128;
constexpr int kCommitBatch = 8;

// One CTA per sequence, layer, keys or values.  Each thread owns one 16-byte
// column of the entries and moves it for all accepted nodes in order, eight at a
// time: the sources of a batch are read before any of its targets is written,
// and since a_i >= i is increasing, no target is the source of a later batch.
// Bound by memory (or, for a few rows, by latency): every moved entry is read
// once and written once.
__global__ void __launch_bounds__(kCommitThreads) kv_commit_kernel(const CommitArgs a) {
    __shared__ long long s_src[kMaxN], s_dst[kMaxN];
    const int b = blockIdx.z, tid = threadIdx.x;
    const Cache& c = a.c;
    const int n = a.num_accepted[b], len = a.kv_len[b];
    const bool first = blockIdx.x == 0 && blockIdx.y == 0 && tid == 0;
    uint32_t bad = 0;
    const long long cap = (long long)c.table_width << c.page_shift;
    if (n < -1 || n >= a.N || len < 0 || (long long)len + n + 1 > cap) {
        bad = SV_DEV_BAD_LENGTH;
    } else if (n > 0 && a.out_nodes) {
        int f = 0;
        if (tid < n) {
            const int32_t* nodes = a.out_nodes + (long long)b * a.N;
            const int x = nodes[tid], before = tid ? nodes[tid - 1] : 0;
            // the last slot within the table bounds them all
            if (x <= before || x >= a.N) {
                f = SV_DEV_BAD_TREE;
            } else if ((long long)len + x >= cap) {
                f = SV_DEV_BAD_LENGTH;
            } else {
                const bool stays = x == tid + 1;
                s_src[tid] = stays ? 0 : slot_offset(c, b, len + x);
                s_dst[tid] = stays ? -1 : slot_offset(c, b, len + tid + 1);
                if (!stays && (s_src[tid] < 0 || s_dst[tid] < 0)) f = SV_DEV_BAD_PAGE;
            }
        }
        bad = __syncthreads_or(f & SV_DEV_BAD_TREE)     ? SV_DEV_BAD_TREE
              : __syncthreads_or(f & SV_DEV_BAD_LENGTH) ? SV_DEV_BAD_LENGTH
              : __syncthreads_or(f)                     ? SV_DEV_BAD_PAGE
                                                        : 0;
    }
    if (first) {
        if (bad) mark(a.status, b, bad);
        a.kv_len_out[b] = bad ? len : len + n + 1;
    }
    if (bad || n <= 0 || !a.out_nodes) return;
    char* base = (blockIdx.y & 1 ? c.v : c.k) + (long long)(blockIdx.y >> 1) * a.layer_stride;
    const int u = blockIdx.x * kCommitThreads + tid;
    if (u >= a.units) return;
    const int h = u / a.head_units;
    base += h * c.head_stride + (u - h * a.head_units) * 16;
    for (int i0 = 0; i0 < n; i0 += kCommitBatch) {
        uint4 x[kCommitBatch];
#pragma unroll
        for (int i = 0; i < kCommitBatch; ++i)
            if (i0 + i < n && s_dst[i0 + i] >= 0)
                x[i] = *reinterpret_cast<const uint4*>(base + s_src[i0 + i]);
#pragma unroll
        for (int i = 0; i < kCommitBatch; ++i)
            if (i0 + i < n && s_dst[i0 + i] >= 0)
                *reinterpret_cast<uint4*>(base + s_dst[i0 + i]) = x[i];
    }
}

// ---------------------------------------------------------------- host

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

static sv_status device_ok() {
    static std::mutex mu;
    static int known[64];  // 0 unknown, 1 sm_103, 2 another device
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SV_ERR_CUDA;
    if (dev < 0 || dev >= 64) return SV_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lk(mu);
    if (!known[dev]) {
        int major = 0, minor = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
            return SV_ERR_CUDA;
        known[dev] = major == 10 && minor == 3 ? 1 : 2;
    }
    return known[dev] == 1 ? SV_OK : SV_ERR_UNSUPPORTED;
}

static int elem_bytes(sv_dtype t) { return t == SV_E4M3 ? 1 : 2; }

// scales: the call needs the scales of a float8 cache.
static sv_status check_cache(const sv_kv_cache* c, bool scales, Cache* out) {
    if (!c || !c->k || !c->v || !c->table) return SV_ERR_INVALID_ARG;
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
static void launch_append(const AppendArgs& a, int B, cudaStream_t s) {
    const dim3 grid(a.N, B);
    // whole 16-byte accesses when the rotated and the remaining part allow it
    if (a.rot % 16 == 0)
        kv_append_kernel<T, CT, 8><<<grid, kAppendThreads, 0, s>>>(a);
    else if (a.rot % 8 == 0)
        kv_append_kernel<T, CT, 4><<<grid, kAppendThreads, 0, s>>>(a);
    else
        kv_append_kernel<T, CT, 1><<<grid, kAppendThreads, 0, s>>>(a);
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
    sv_status st = check_cache(cache, true, &a.c);
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
    if ((st = device_ok()) != SV_OK) return st;
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
            launch_append<__nv_bfloat16, __nv_fp8_e4m3>(a, B, stream);
        else
            launch_append<__nv_bfloat16, __nv_bfloat16>(a, B, stream);
    } else {
        if (cache->dtype == SV_E4M3)
            launch_append<__half, __nv_fp8_e4m3>(a, B, stream);
        else
            launch_append<__half, __half>(a, B, stream);
    }
    return launched();
}

size_t spec_kv_attention_workspace_size(int B, int N, int q_heads, int heads, int dim) {
    if (B < 0 || B > kMaxB || N < 1 || N > kMaxN || heads < 1 || q_heads < 1 || q_heads % heads ||
        q_heads > kMaxQHeads || dim < 16 || dim > kMaxDim || dim % 16)
        return 0;
    return 256;
}

sv_status spec_kv_attention(const sv_kv_cache* cache, const void* q, const sv_strides* q_strides,
                            sv_dtype dtype, const int32_t* kv_len, const int32_t* num_new,
                            const int32_t* tree_parents, float scale, int B, int N, int q_heads,
                            void* out, void* ws, size_t ws_bytes, uint32_t* status,
                            cudaStream_t stream) {
    AttentionArgs a = {};
    sv_status st = check_cache(cache, true, &a.c);
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
    if ((st = device_ok()) != SV_OK) return st;
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
    const dim3 grid(q_heads, N, B);
    if (dtype == SV_BF16) {
        if (cache->dtype == SV_E4M3)
            kv_attention_kernel<__nv_bfloat16, __nv_fp8_e4m3><<<grid, kSimpleThreads, 0, stream>>>(a);
        else
            kv_attention_kernel<__nv_bfloat16, __nv_bfloat16><<<grid, kSimpleThreads, 0, stream>>>(a);
    } else {
        if (cache->dtype == SV_E4M3)
            kv_attention_kernel<__half, __nv_fp8_e4m3><<<grid, kSimpleThreads, 0, stream>>>(a);
        else
            kv_attention_kernel<__half, __half><<<grid, kSimpleThreads, 0, stream>>>(a);
    }
    return launched();
}

sv_status spec_kv_commit(const sv_kv_cache* cache, int layers, int64_t layer_stride,
                         const int32_t* kv_len, const int32_t* out_nodes,
                         const int32_t* num_accepted, int B, int N, int32_t* kv_len_out,
                         uint32_t* status, cudaStream_t stream) {
    CommitArgs a = {};
    sv_status st = check_cache(cache, false, &a.c);
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
    if (kv_len_out == kv_len) return SV_ERR_INVALID_ARG;
    if ((st = device_ok()) != SV_OK) return st;
    a.layer_stride = layers > 1 ? layer_stride * e : 0;
    a.kv_len = kv_len;
    a.out_nodes = out_nodes;
    a.num_accepted = num_accepted;
    a.kv_len_out = kv_len_out;
    a.status = status;
    a.N = N;
    a.head_units = cache->dim * e / 16;
    a.units = cache->heads * a.head_units;
    const dim3 grid((a.units + kCommitThreads - 1) / kCommitThreads, 2 * layers, B);
    kv_commit_kernel<<<grid, kCommitThreads, 0, stream>>>(a);
    return launched();
}

}  // extern "C"
