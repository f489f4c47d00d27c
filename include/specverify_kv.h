/*
 * specverify_kv — what a speculative round does to the target's paged
 * key-value cache, on one GB300 (sm_103a), behind the same plain C ABI as
 * specverify.h.
 *
 * A round drafts N tokens per sequence (a chain, or a tree as for
 * spec_verify_tree: node 0 is the last committed token, whose own entry is not
 * cached yet).  In every layer the target rotates their queries and keys to
 * their positions and writes keys and values behind the cached ones
 * (spec_kv_append), and lets every drafted token attend to the cached
 * positions and to its own ancestors (spec_kv_attention: the tree-attention
 * pass that produces the logits rows which spec_verify_* judges).  After the
 * verdict the accepted nodes' entries move up behind the committed ones in
 * every layer, and the rest is dropped (spec_kv_commit: "Decodificação
 * especulativa explicada: rascunhe barato, verifique numa passada", §"O ciclo de
 * rascunho e verificação", bookkeeping paragraph; "Speculative decoding: el
 * secretario que adelanta lo que va a decir el jefe", §"Tree attention").  With
 * N = 1 append and attention are one step of plain decoding.
 *
 * Slots.  kv_len[b] counts the committed entries of sequence b; all three calls
 * of a round take the same kv_len.  Node j's entry is in slot kv_len[b] + j
 * (slot s is entry s % page_size of page table[b][s / page_size]); its position
 * is kv_len[b] + depth(j), depth 0 at the root.  After commit the accepted nodes
 * a_1 < ... < a_n are in slots kv_len[b] + 1 .. kv_len[b] + n and kv_len_out[b] =
 * kv_len[b] + n + 1 (the root and the accepted nodes), as spec_verify_*_kv
 * counts.
 *
 * Conventions beyond those of specverify.h (device pointers, 16-byte alignment,
 * asynchronous launches, argument errors before any launch, no allocation).
 *  - tree_parents [B, N] int32 as for spec_verify_tree (entry 0 unused), or NULL
 *    for a chain (node j's parent is j - 1).
 *  - num_new [B] int32 or NULL: the tokens that sequence b really has (its first
 *    num_new[b] of N); NULL: N each.  Rows behind them are left as they were.
 *  - status [B] uint32 or NULL: SV_DEV_* bits are ORed into it atomically; the
 *    caller zeroes it when it wants fresh bits.  Bad data found on the device:
 *      SV_DEV_BAD_LENGTH  kv_len negative, num_new outside [0, N], or
 *                         kv_len + num_new beyond table_width * page_size;
 *      SV_DEV_BAD_TREE    a parent outside [0, j) at a node j < num_new;
 *      SV_DEV_BAD_PAGE    a page that the call needs outside [0, num_pages).
 *    No memory is read or written through them; what the sequence then gets is
 *    said at each call.  Table entries that a call does not need are not read.
 *  - Several sequences may share pages of their committed slots; the pages that
 *    append and commit write belong to one sequence each.
 *  - Limits: 1 <= N <= 65, B <= 65535, dim a multiple of 16 up to 128,
 *    page_size a power of two, table_width * page_size < 2^31, q_heads a
 *    multiple of heads and at most 1024.  B == 0 launches nothing.
 */
#ifndef SPECVERIFY_KV_H
#define SPECVERIFY_KV_H

#include "specverify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Types of queries, new keys and values, and caches (sv_dtype values beside
 * SV_BF16; the logits calls of specverify.h do not take them). */
#define SV_F16 ((sv_dtype)2)
#define SV_E4M3 ((sv_dtype)3) /* caches only: 8-bit floating point, 4 exponent bits */

#define SV_DEV_BAD_PAGE 0x80u
#define SV_DEV_BAD_LENGTH 0x100u
#define SV_DEV_TIMEOUT 0x200u /* spec_kv_attention: a bounded wait inside the kernel gave up */

/* One layer of a paged cache.  Entry (page p, slot s, head h) starts at element
 * p*page_stride + s*slot_stride + h*head_stride of k and of v, its dim elements
 * contiguous, so that pages may hold slots of heads or heads of slots.  Strides
 * are in elements, positive and multiples of 16 bytes. */
typedef struct {
    void* k;                /* DEVICE */
    void* v;                /* DEVICE */
    const int32_t* table;   /* DEVICE [B, table_width]: the pages of each sequence; */
                            /* may be NULL if B is 0                            */
    const float* k_scale;   /* DEVICE [heads], SV_E4M3 only (NULL otherwise):   */
    const float* v_scale;   /* an entry stands for its stored value times this, */
                            /* of either sign; spec_kv_commit does not look at  */
                            /* them                                             */
    int64_t page_stride, slot_stride, head_stride;
    int num_pages, page_size, table_width;
    int heads, dim;
    sv_dtype dtype;         /* SV_BF16, SV_F16 or SV_E4M3 */
} sv_kv_cache;

/* Strides, in elements, of a [B, N, heads, dim] tensor whose dim elements are
 * contiguous: multiples of 16 bytes, so that queries, keys and values may be
 * slices of one projection's output. */
typedef struct {
    int64_t batch, token, head;
} sv_strides;

/* A rotation of the first rot_dim elements of each head by the position: pair i
 * = elements (i, i + rot_dim/2), or (2i, 2i + 1) when interleaved, becomes
 * magnitude * (a cos - b sin, b cos + a sin) of position * rate_i.  turns holds
 * the rates in turns per position as 64-bit binary fractions, so that position *
 * rate modulo one turn is exact integer arithmetic at any position. */
typedef struct {
    const uint64_t* turns;  /* DEVICE [rot_dim / 2], from spec_kv_rope_turns */
    int rot_dim;            /* even, 2 <= rot_dim <= dim */
    int interleaved;
    float magnitude;        /* 1: a plain rotation */
} sv_rope;

/* Fills turns (HOST, rot_dim/2 entries) with rate_i = base^(-2i/rot_dim) / 2pi,
 * scaled for contexts `factor` times the trained length: with original_length
 * <= 0 every rate is divided by factor; otherwise a pair that makes at least
 * `high` turns over the original length keeps its rate, one that makes at most
 * `low` has it divided by factor, and between them the two are mixed linearly in
 * the number of turns.  factor 1 leaves the rates alone.  SV_ERR_INVALID_ARG
 * unless base > 1, factor >= 1 and low < high, all finite. */
sv_status spec_kv_rope_turns(int rot_dim, double base, double factor, double original_length,
                             double low, double high, uint64_t* turns);

/* Rotates the N new tokens' queries and keys and writes keys and values into
 * the cache.
 *   k, v    [B, N, heads, dim] of type dtype (SV_BF16 or SV_F16), strides
 *           kv_strides; the cache has the same type, or SV_E4M3: the entry
 *           divided by the head's scale, rounded to nearest, saturating.
 *   q       [B, N, q_heads, dim], strides q_strides, or NULL (keys and values
 *           only; q_heads, q_strides and q_out are then ignored).
 *   q_out   [B, N, q_heads, dim] contiguous (written): q rotated.  It may be q
 *           itself when q is contiguous; otherwise it must not overlap it.
 *   rope    NULL: nothing is rotated.  The arithmetic is fp32, rounded once.
 * A sequence with a bad length or tree is left alone entirely; a token with a
 * bad page gets q_out but no entry. */
sv_status spec_kv_append(const sv_kv_cache* cache, const sv_rope* rope, const void* q,
                         const sv_strides* q_strides, const void* k, const void* v,
                         const sv_strides* kv_strides, sv_dtype dtype, const int32_t* kv_len,
                         const int32_t* num_new, const int32_t* tree_parents, int B, int N,
                         int q_heads, void* q_out, uint32_t* status, cudaStream_t stream);

/* Bytes of workspace of spec_kv_attention (0 for invalid sizes). */
size_t spec_kv_attention_workspace_size(int B, int N, int q_heads, int heads, int dim);

/* Attention of the N new tokens (whose entries are in the cache) over the paged
 * cache: out_j = sum_l p_jl v_l, p_j = softmax over l of scale * q_j . k_l, l
 * running over the committed slots and over the slots of node j and its
 * ancestors.  Query head h reads key head h / (q_heads / heads).
 *   q    [B, N, q_heads, dim], SV_BF16 or SV_F16, strides q_strides; the cache
 *        has the same type, or SV_E4M3.
 *   out  [B, N, q_heads, dim] contiguous (written), the type of q; it must not
 *        overlap q.
 * Entries that a node does not attend to take no part, whatever they hold.
 * Workspace as for the other calls (no initialisation; calls that share one must
 * not overlap).  Every row of a sequence with a bad length, tree or page, or of a
 * wait that gave up (SV_DEV_TIMEOUT), is NaN (its first num_new rows; all N when
 * num_new itself is bad).
 *
 * Arithmetic.  Scores, maxima and sums are fp32; the products are the tensor
 * cores', of 16-bit operands with fp32 sums.
 *  - The weights are multiplied as two 16-bit halves (hi + lo), which leaves
 *    nothing of their rounding, with at most 32 query rows (N * q_heads / heads)
 *    per key head, unless the cache is SV_E4M3 and q SV_BF16.  There, and with
 *    more rows, they are rounded once to 16 bits: that of q's type, fp16 over
 *    SV_E4M3.
 *  - In fp16, weights below 2^-25 of the largest so far are missing in the output
 *    but not in the sum that it is divided by.
 *  - The tensor cores' sums cut off, rather than round, what lies below about
 *    2^-24 of the running sum, so that many faint slots beside one that holds most
 *    of the weight lose part of theirs, in every type: up to 0.2 % of the result
 *    with 131072 of them, up to 0.8 % with 524288 (measured, 264 rows per key
 *    head; a quarter of it with few rows).
 *  - SV_BF16 queries over an SV_E4M3 cache become halves, after a power of two per
 *    row has been taken out: exact down to 2^-25 of the row's largest element, and
 *    zero below 2^-34 of it.
 *
 * The form is chosen from the sizes and types alone, the longest context being
 * what the table has room for (table_width * page_size): one with no more room
 * than its batch needs may be faster (one token over 700 slots: 5.7 us where there
 * is room for at most 8192, 9.1 us beyond). */
sv_status spec_kv_attention(const sv_kv_cache* cache, const void* q, const sv_strides* q_strides,
                            sv_dtype dtype, const int32_t* kv_len, const int32_t* num_new,
                            const int32_t* tree_parents, float scale, int B, int N, int q_heads,
                            void* out, void* ws, size_t ws_bytes, uint32_t* status,
                            cudaStream_t stream);

/* After verification: moves the accepted nodes' entries of `layers` layers
 * (layer i's keys and values at k and v + i*layer_stride elements; layer_stride
 * a multiple of 16 bytes, ignored for one layer) to the slots behind the root's
 * and writes the new lengths.
 *   out_nodes     [B, N] int32: the accepted nodes in order, as spec_verify_tree
 *                 writes them, or NULL for a chain (nothing moves).
 *   num_accepted  [B] int32: how many of them; -1 (an invalid sequence): nothing
 *                 moves and kv_len_out = kv_len.
 *   kv_len_out    [B] int32 (written): kv_len + num_accepted + 1.  Must not
 *                 overlap kv_len or num_accepted.
 * A sequence whose accepted nodes are not increasing within [1, N)
 * (SV_DEV_BAD_TREE), whose num_accepted is outside [-1, N - 1] or whose slots
 * lie beyond the table (SV_DEV_BAD_LENGTH) or that needs a bad page stays as it
 * is, kv_len_out = kv_len. */
sv_status spec_kv_commit(const sv_kv_cache* cache, int layers, int64_t layer_stride,
                         const int32_t* kv_len, const int32_t* out_nodes,
                         const int32_t* num_accepted, int B, int N, int32_t* kv_len_out,
                         uint32_t* status, cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* SPECVERIFY_KV_H */
