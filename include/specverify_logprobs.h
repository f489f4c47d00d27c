/*
 * specverify_logprobs — log probabilities of given tokens, with the entropy and
 * the most probable alternatives of their rows, and the gradient of both to the
 * logits; on one GB300 (sm_103a), behind the same plain C ABI as specverify.h.
 *
 * The rows are those that spec_verify_* judges: p = softmax(l / T) of the
 * target's logits [B, k+1, V], asked about out_tokens after the verdict (what a
 * server tells its user beside a round's tokens), or the draft's own logits
 * asked about the target's alternatives (what a draft is trained on while it
 * serves).
 *
 * With m = max_v l_v, S = sum_v exp((l_v - m) / T):
 *   log p_v = (l_v - m) / T - ln S,      H = -sum_v p_v ln p_v.
 *
 * Conventions beyond those of specverify.h (device pointers, asynchronous
 * launches, argument errors before any launch, no allocation).
 *  - A call takes `rows` rows of V logits, row_stride elements apart (at least
 *    V, any number: rows need not begin on a 16-byte boundary; the first does).
 *  - tokens [rows, given] int32: the tokens asked about in each row, in any
 *    order, the same one more than once or not; -1 where there is none (as
 *    out_tokens behind the emitted token).  A row without any is not read, and
 *    what belongs to it is left as it was (its gradient: zeros).  1 <= given <=
 *    64.
 *  - status [rows] uint32 or NULL: SV_DEV_* bits are ORed into it atomically;
 *    the caller zeroes it when it wants fresh bits.
 *      SV_DEV_BAD_ROW    a NaN or +inf among the row's logits, or all are -inf;
 *      SV_DEV_BAD_TOKEN  a token below -1 or not below V.
 *  - Limits: V <= 2^21, rows < 2^27, rows * row_stride < 2^40, T from 2^-100 to
 *    2^100.  rows == 0 launches nothing.
 *  - The arithmetic is fp32, whatever the type of the logits; results repeat bit
 *    for bit.
 */
#ifndef SPECVERIFY_LOGPROBS_H
#define SPECVERIFY_LOGPROBS_H

#include "specverify.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SV_LOGPROBS_MAX_GIVEN 64
#define SV_LOGPROBS_MAX_TOP 64

/* Bytes of workspace of spec_logprobs (0 for invalid sizes). */
size_t spec_logprobs_workspace_size(int rows, int V, sv_dtype dtype, int given, int top);

/* Log probabilities, entropy and alternatives.
 *   logits        [rows, V] bf16 or fp32 (dtype), rows row_stride apart.
 *   T             temperature, finite and > 0.
 *   logprobs      [rows, given] fp32 (written where tokens holds one): ln p of it;
 *                 -inf for a token whose logit is -inf.
 *   normalizer    [rows, 2] fp32 (written) or NULL: m and ln S, which
 *                 spec_logprobs_grad takes.
 *   entropy       [rows] fp32 (written) or NULL: H.
 *   top_tokens    [rows, top] int32 (written), 0 <= top <= 64: the tokens with
 *                 the largest logits, largest first, the lower token first among
 *                 equals; -1 behind V of them.  NULL when top is 0.
 *   top_logprobs  [rows, top] fp32 (written): their ln p; -inf behind V of them.
 * A bad row gets NaN everywhere (top_tokens -1), a bad token NaN at its own place.
 * The workspace is asked for as by the verify calls (spec_logprobs_workspace_size bytes
 * at least, 16-byte aligned) but neither read nor written: calls that overlap, and
 * captured graphs, may share one.
 * Accuracy: a weight's exponent is off by the rounding of l - m and its own, 2^-24
 * |l - m| / T each, the exponential by 2^-21 besides, and the sums by the fp32
 * additions of a thread's share.  Against 64 bits, in rows of 2^18 tokens like a
 * model's, ln p is off by 3e-6 at most (2^-20 for each of two roundings where it is
 * below -16) and H by 1.5e-6; where many nearly equal elements weigh as much as the
 * large ones, 2e-6 and 7e-6 (rows of 2^21: 6e-6 and 2e-5).  Alternatives are told
 * apart by their exact values. */
sv_status spec_logprobs(const void* logits, sv_dtype dtype, int64_t row_stride,
                        const int32_t* tokens, float T, int rows, int V, int given, int top,
                        float* logprobs, float* normalizer, float* entropy, int32_t* top_tokens,
                        float* top_logprobs, void* ws, size_t ws_bytes, uint32_t* status,
                        cudaStream_t stream);

/* The gradient to the logits of sum_j grad_logprobs_j ln p(token_j) + grad_entropy H:
 *   dl_v = (sum_j g_j (1[v = token_j] - p_v) - g_H p_v (ln p_v + H)) / T,
 * rounded once to the type of the logits.
 *   normalizer    [rows, 2], entropy [rows]: as spec_logprobs wrote them for these
 *                 logits and this T.
 *   grad_logprobs [rows, given] fp32 (not looked at where tokens holds none).
 *   grad_entropy  [rows] fp32, or NULL (entropy is then ignored and may be NULL).
 *   grad_logits   [rows, V] of the type of the logits (written: every row), rows
 *                 grad_stride apart.  It may be logits itself when the strides are
 *                 equal; otherwise it must not overlap it.
 * A row with a bad token or a normalizer that is not finite becomes NaN. */
sv_status spec_logprobs_grad(const void* logits, sv_dtype dtype, int64_t row_stride,
                             const int32_t* tokens, const float* normalizer, const float* entropy,
                             const float* grad_logprobs, const float* grad_entropy, float T,
                             int rows, int V, int given, void* grad_logits, int64_t grad_stride,
                             uint32_t* status, cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* SPECVERIFY_LOGPROBS_H */
