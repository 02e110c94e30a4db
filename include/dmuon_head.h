/*
 * libdmuon_ns -- losses of a language model's output head and their gradients,
 * C ABI.  The head is the matrix whose gradient the AdamW step of dmuon_ns.h
 * takes next; these calls produce that gradient without ever holding the
 * tokens x vocab logits.
 *
 * With hidden states H (tokens x hidden) and the head's weight W (vocab x
 * hidden), s = H W^T (each product of two inputs exact, summed in fp32):
 *
 *   softmax cross entropy
 *     lse_t  = log sum_v exp(s_tv),   loss_t = lse_t - s_t,target(t)
 *     ds_tv  = (g_t + gl_t) p_tv - g_t [v = target(t)],  p_tv = exp(s_tv - lse_t)
 *   distillation from a teacher's top logits, at temperature T
 *     q_tk   = softmax of z_tk / T over the row's entries (ids[t][k] >= 0)
 *     lse_t  = log sum_v exp(s_tv / T)
 *     loss_t = T^2 sum_k q_tk (log q_tk - s_t,id(t,k) / T + lse_t)
 *     ds_tv  = T g_t (p_tv - sum of q_tk with id(t,k) = v),  p_tv = exp(s_tv / T - lse_t)
 *   both:  dH = ds W,  dW = ds^T H
 *
 * g_t is the upstream gradient of loss_t, gl_t that of lse_t (a penalty on the
 * normaliser, for example).  The vocabulary is worked through in pieces; the
 * backward call computes each piece's s again.
 *
 * Rows that carry no loss -- the target is ignore_index, or no teacher entry
 * has an id >= 0 and a logit above -inf -- have loss_t = lse_t = 0 and take no
 * part in any product: their rows of dH are 0 and whatever their rows of H
 * hold (NaN included) reaches nothing.  A target outside [0, vocab) that is
 * not ignore_index, or a teacher id >= vocab, makes the row's loss NaN and the
 * gradients NaN (dW too): nothing outside the arrays is ever read or written.
 * A teacher entry whose logit is -inf has no mass and its id is not held against
 * the row: from vocab on it is passed over like an absent one (student_logits 0).
 * A NaN or +inf logit of a present entry makes the row's loss NaN.
 *
 * Arithmetic.  Sums and softmax statistics are fp32.  A loss is formed from the
 * distances of logits, not from lse.  A probability is exp(s / T - lse) with lse
 * rounded to fp32, so it is good to about 2^-24 (1 + |lse|) relative.  Entries of ds
 * below 2^-126 of the largest gradient weight count as 0.  Teacher logits may hold
 * fp32's lowest value (equal ones share the row's mass) and -inf (no mass).
 *
 * DMUON_BF16: bf16 operands.  ds is rounded to bf16 once as the operand of its two
 * products, relative to the largest gradient weight (gradients are then off by 1.1
 * to 1.4 times what rounding them to bf16 alone costs); in calls of at most 128
 * tokens, ignored ones included, it is held in two bf16 parts (16 bits).
 *
 * DMUON_F32: operands are multiplied in parts.  Gradients, and the logits of few
 * tokens (forward up to 256, backward up to 384, ignored ones included): three bf16
 * parts that hold all 24 bits.  Logits otherwise: two fp16 parts of rows scaled by a
 * power of two; a logit is off by at most 2^-21 of the sum of its products'
 * magnitudes, and by 2^-22 T more where a row's elements differ by more than 2^17.
 * Calls whose rows could make that more take the three parts, at up to three times
 * the time of the logits' product: decided on the device, where the largest |h|
 * times the largest sum of a row of |W|, plus the same the other way round, is above
 * 2^17 T.  Inputs of magnitude up to 3e38; elements below 2^-108 lose their last
 * bits.
 *
 * Conventions are those of dmuon_ns.h: status codes, dense row-major arrays,
 * 16-byte aligned device pointers of the current device, a 256-byte aligned
 * workspace of the caller's, arguments checked before anything is enqueued, no
 * written buffer overlapping another one of the call, nothing allocated or
 * synchronised (calls may be captured in a HIP graph), deterministic results.
 * Calls that share a workspace must not overlap in time; nothing needs to stay
 * in it between calls.
 */
#ifndef DMUON_HEAD_H
#define DMUON_HEAD_H

#include "dmuon_ns.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Sizes of a head loss.  0 <= tokens < 2^24, 1 <= hidden <= 65536, 1 <= vocab
 * < 2^27, tokens x vocab <= 2^42, 0 <= top_k <= 1024 (teacher entries a token;
 * 0 for cross entropy).
 * dtype (dmuon_dtype): of H and W and of their gradients. */
typedef struct {
    int64_t tokens;
    int64_t hidden;
    int64_t vocab;
    int32_t top_k;
    int32_t dtype;
} dmuon_head_desc;

/* Bytes of device workspace that serve every forward (backward == 0) or
 * backward call of at most these tokens and these other sizes.  Errors: INVALID_ARG (null
 * pointer, a size out of the ranges above below its minimum, unknown dtype),
 * UNSUPPORTED (a size above its maximum). */
DMUON_API dmuon_status head_loss_workspace_bytes(const dmuon_head_desc* desc, int32_t backward, size_t* bytes);

/* Softmax cross entropy, forward (desc->top_k 0).
 *   hidden  device, tokens x hidden, dtype      weight  device, vocab x hidden, dtype
 *   targets device, tokens int64                losses, lse  device, tokens fp32, written
 * tokens == 0 is a no-op.  Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE, ALLOC, HIP. */
DMUON_API dmuon_status head_cross_entropy_forward(const dmuon_head_desc* desc, const void* hidden, const void* weight,
                                                  const int64_t* targets, int64_t ignore_index, float* losses,
                                                  float* lse, void* workspace, size_t workspace_bytes, void* stream);

/* Softmax cross entropy, backward.  lse is the forward call's; grad_losses and
 * grad_lse (NULL: zero) are tokens fp32, not read where the target is
 * ignore_index.  grad_hidden (tokens x hidden) and grad_weight (vocab x hidden)
 * are overwritten; either may be NULL and is then not computed (not both).
 * tokens == 0 fills grad_weight with zeros. */
DMUON_API dmuon_status head_cross_entropy_backward(const dmuon_head_desc* desc, const void* hidden,
                                                   const void* weight, const int64_t* targets, int64_t ignore_index,
                                                   const float* lse, const float* grad_losses, const float* grad_lse,
                                                   void* grad_hidden, void* grad_weight, void* workspace,
                                                   size_t workspace_bytes, void* stream);

/* Distillation, forward (desc->top_k >= 1).  teacher_ids int64 and
 * teacher_logits fp32 are tokens x top_k; an entry with id < 0 is absent and
 * its logit is not used.  An id may repeat in a row: its entries' q add up in
 * the gradient.  student_logits (tokens x top_k fp32, written) receives
 * s_t,id(t,k), 0 for absent entries and rows without loss; the backward call
 * takes it.  temperature is > 0 with a normal fp32 square (1.1e-19 to 1.8e19);
 * a loss is good to about T^2 2^-24 times its largest term (log q, log vocab, the
 * distance of s from the row's largest logit over T), beside its logits' error. */
DMUON_API dmuon_status head_distill_forward(const dmuon_head_desc* desc, const void* hidden, const void* weight,
                                            const int64_t* teacher_ids, const float* teacher_logits,
                                            float temperature, float* losses, float* lse, float* student_logits,
                                            void* workspace, size_t workspace_bytes, void* stream);

/* Distillation, backward: as head_cross_entropy_backward, with the forward
 * call's lse and student_logits. */
DMUON_API dmuon_status head_distill_backward(const dmuon_head_desc* desc, const void* hidden, const void* weight,
                                             const int64_t* teacher_ids, const float* teacher_logits,
                                             float temperature, const float* lse, const float* student_logits,
                                             const float* grad_losses, void* grad_hidden, void* grad_weight,
                                             void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DMUON_HEAD_H */
