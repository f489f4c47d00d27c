// The paged key-value cache of a speculative round: append with rotation,
// attention of the drafted tokens, commit of the accepted ones
// (include/specverify_kv.h).

#include "kvattention.cuh"

namespace svkv {

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
    return attend<false>(cache, q, q_strides, dtype, kv_len, num_new, tree_parents, scale, 0, 0, B,
                         N, q_heads, out, ws, ws_bytes, status, stream);
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
