/*
 * libdmuon_ns -- log probabilities of given tokens over a language model's
 * output head, with the entropy and the most likely alternatives of each
 * token's distribution, and their gradients, C ABI.  What a policy gradient,
 * scoring or a teacher's pass takes from the head, without ever holding the
 * tokens x vocab logits of a large vocabulary.
 *
 * With hidden states H (tokens x hidden), the head's weight W (vocab x hidden)
 * and a temperature T, s = H W^T (each product of two inputs exact, summed in
 * fp32) and x = s / T:
 *
 *   lse_t     = log sum_v exp x_tv                p_tv = exp(x_tv - lse_t)
 *   logprob_t = x_t,target(t) - lse_t
 *   entropy_t = - sum_v p_tv log p_tv
 *   alternatives: the K largest s_tv of the row in descending order, equal ones
 *     by the lower id, with x_tv - lse_t
 *   gradient of sum_t (g_t logprob_t + e_t entropy_t):
 *     dx_tv = g_t ([v = target(t)] - p_tv) - e_t p_tv (x_tv - lse_t + entropy_t)
 *     dH = dx W / T,  dW = dx^T H / T
 *
 * The alternatives' values carry no gradient.  top_logprobs of T = 1 are what
 * head_distill_forward takes as teacher_logits, with top_ids as teacher_ids.
 *
 * Rows whose target is ignore_index take no part in any product: logprob_t,
 * entropy_t, lse_t and their alternatives' values are 0, the alternatives' ids
 * -1, their rows of dH 0, and whatever their rows of H hold (NaN included)
 * reaches nothing.  A target outside [0, vocab) that is not ignore_index makes
 * logprob_t NaN (the row's other outputs stand) and the gradients NaN (dW too).
 * Without targets (NULL) every row counts and there are no logprobs.
 *
 * A row with a logit that is NaN or +inf, or with none above -inf, has NaN
 * outputs and -1 as its alternatives' ids.  Where fewer than K logits are above
 * -inf the further alternatives have id -1 and value -inf.  Terms of the entropy
 * with p = 0 are 0.  Words are masked by weights that make their logits low: finite
 * ones, of the type's lowest value in bf16 and of magnitude up to 3e38 in fp32, whose
 * logits may overflow to -inf; in bf16's forward calls also -inf.  (dH is dx W: an
 * infinite weight makes it NaN where dx is 0.  fp32 inputs are multiplied in parts, which
 * neither an infinity nor fp32's lowest value has: one in H or W makes the rows that
 * it meets NaN.)
 *
 * Arithmetic as in dmuon_head.h: sums and softmax statistics are fp32; log
 * probabilities and entropies are formed from the distances of logits from the
 * row's largest one, not from lse; ds in the gradients' products is held as there
 * (bf16 calls round it to bf16 once, relative to the largest of |g|, |e| and
 * |g + e entropy|; entries below 2^-126 of that count as 0), fp32 calls multiply in
 * parts.  An alternative is found by the logit that its product formed; where several of
 * a row's alternatives lie in one group of 16 words, all but the first of them are by
 * logits formed again in another order of summation, which may differ in the last bits
 * and so order what those bits decide otherwise.  How sums are cut follows from the
 * call's sizes, so a row's last bits may differ between calls of other sizes; a call with
 * alternatives takes as many tokens at a time as 1 GiB holds what it keeps of them.
 *
 * Conventions are those of dmuon_head.h: status codes, dense row-major arrays,
 * 16-byte aligned device pointers of the current device, a 256-byte aligned
 * workspace of the caller's, arguments checked before anything is enqueued, no
 * written buffer overlapping another one of the call, nothing allocated or
 * synchronised (calls may be captured in a HIP graph), deterministic results.
 * Calls that share a workspace must not overlap in time; nothing needs to stay
 * in it between calls.
 */
#ifndef DMUON_LOGPROBS_H
#define DMUON_LOGPROBS_H

#include "dmuon_head.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Sizes as for a head loss (dmuon_head_desc: tokens, hidden, vocab, dtype);
 * top_k is K, the alternatives a token: 0 <= top_k <= 128 and <= vocab forward,
 * 0 backward. */

/* Bytes of device workspace that serve every forward (backward == 0) or
 * backward call of at most these tokens and these other sizes.  Errors:
 * INVALID_ARG (null pointer, a size out of its range above or below its
 * minimum, unknown dtype), UNSUPPORTED (a size above its maximum). */
DMUON_API dmuon_status head_log_probs_workspace_bytes(const dmuon_head_desc* desc, int32_t backward, size_t* bytes);

/* Forward.
 *   hidden  device, tokens x hidden, dtype      weight  device, vocab x hidden, dtype
 *   targets device, tokens int64, or NULL       logprobs device, tokens fp32 (NULL with targets, and only then)
 *   entropy device, tokens fp32, or NULL        lse  device, tokens fp32
 *   top_ids device, tokens x top_k int64, top_logprobs device, tokens x top_k fp32 (both NULL for top_k == 0)
 * temperature is a normal fp32 number > 0 with a normal inverse.  tokens == 0 is
 * a no-op.  Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, ALLOC, HIP. */
DMUON_API dmuon_status head_log_probs_forward(const dmuon_head_desc* desc, const void* hidden, const void* weight,
                                              const int64_t* targets, int64_t ignore_index, float temperature,
                                              float* logprobs, float* entropy, float* lse, int64_t* top_ids,
                                              float* top_logprobs, void* workspace, size_t workspace_bytes,
                                              void* stream);

/* Backward.  lse and entropy are the forward call's (entropy may be NULL where
 * grad_entropy is); grad_logprobs and grad_entropy are tokens fp32, not read
 * where the target is ignore_index; either may be NULL and counts as zeros (not
 * both), grad_logprobs has to be where targets is.  grad_hidden (tokens x
 * hidden) and grad_weight (vocab x hidden), of desc's dtype, are overwritten;
 * either may be NULL and is then not computed (not both).  tokens == 0 fills
 * grad_weight with zeros. */
DMUON_API dmuon_status head_log_probs_backward(const dmuon_head_desc* desc, const void* hidden, const void* weight,
                                               const int64_t* targets, int64_t ignore_index, float temperature,
                                               const float* lse, const float* entropy, const float* grad_logprobs,
                                               const float* grad_entropy, void* grad_hidden, void* grad_weight,
                                               void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DMUON_LOGPROBS_H */
