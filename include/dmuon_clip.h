/*
 * libdmuon_ns -- the global norm of many gradients and clipping by it, C ABI.
 *
 *   norm    = sqrt(sum over all elements g of all tensors of g^2)
 *   clipped = g min(1, max_norm / (norm + eps))
 *
 * The two calls are apart so that owners of different tensors can join their
 * norms in between (the norm of all is the root of the sum of their squares).
 * The norm stays on the device: nothing waits for it on the host.
 *
 * Tensors are dense runs of numels[i] elements (0: skipped) of dtypes[i]
 * (DMUON_F32 | DMUON_BF16) that may begin at any element: views into one flat
 * gradient buffer need no padding.  The arrays are host arrays of `count`
 * entries.
 *
 * Arithmetic.  Squares and their sums are formed in 64 bits, in a fixed order:
 * the norm is right to fp32's last place or the one before, neither overflows
 * nor underflows where it is itself a normal fp32 number, and is the same from
 * call to call.  Which tensors follow which decides the order of the sums, so
 * another order of the same tensors may change the last place.  The factor is formed in 64 bits
 * and rounded to fp32; a clipped element is one fp32 product, rounded once more
 * as bf16.
 *
 * NaN and Inf are not masked.  A NaN element makes the norm NaN, and a NaN
 * norm makes every clipped element NaN; an infinite norm makes the factor 0:
 * finite elements become 0, infinite ones NaN.
 *
 * Conventions are those of dmuon_ns.h otherwise: status codes, device pointers
 * of the current device, a 256-byte aligned workspace of the caller's, arguments
 * checked before anything is enqueued, nothing allocated or synchronised (calls
 * may be captured in a HIP graph), deterministic results.  Calls that share a
 * workspace must not overlap in time; nothing needs to stay in it between calls.
 */
#ifndef DMUON_CLIP_H
#define DMUON_CLIP_H

#include "dmuon_ns.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of device workspace for grad_norm_batched over these tensors.  Errors:
 * INVALID_ARG (null pointer, negative count or size, unknown dtype),
 * UNSUPPORTED (2^45 bytes or more in a tensor, or in up to 192 that follow one
 * another). */
DMUON_API dmuon_status grad_norm_workspace_bytes(int32_t count, const int64_t* numels, const int32_t* dtypes,
                                                 size_t* bytes);

/* norm[0] (device, fp32, 4-byte aligned) receives the norm of all tensors; 0 for
 * none.  grads are read only and may overlap one another (elements given twice
 * count twice).  Errors: those above, INVALID_ARG also for a gradient that is
 * null or not aligned to its element and for a norm or workspace that overlaps
 * a gradient or each other; WORKSPACE, HIP, ALLOC. */
DMUON_API dmuon_status grad_norm_batched(int32_t count, const int64_t* numels, const int32_t* dtypes,
                                         const void* const* grads, float* norm, void* workspace,
                                         size_t workspace_bytes, void* stream);

/* outs[i] receives the clipped grads[i], by the norm in norm[0] (device, read
 * only).  outs[i] == grads[i] clips in place, and then nothing is read or
 * written where the factor is 1; any other overlap of an output with another
 * buffer of the call is INVALID_ARG.  max_norm is >= 0 (infinite: nothing is
 * clipped, unless the norm is NaN), eps > 0 and finite.  Errors: as for the
 * norm; INVALID_ARG for max_norm or eps out of range. */
DMUON_API dmuon_status grad_clip_batched(int32_t count, const int64_t* numels, const int32_t* dtypes,
                                         const void* const* grads, void* const* outs, const float* norm,
                                         double max_norm, double eps, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DMUON_CLIP_H */
