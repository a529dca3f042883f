/*
 * moe_distill.h -- the loss that tunes a quantised model (its router, its
 * adapters) towards the unquantised one: the divergence of the logits from a
 * teacher's top logits, and its gradient.
 *
 * For row t with logits z[0 .. V) and the teacher's k entries (id_j, a_j), of which
 * those with id_j in [0, V) are kept:
 *   p_j = exp(a_j / tau) / sum over kept i of exp(a_i / tau)
 *   m = max_v z_v,  l = log sum_v exp((z_v - m) / tau)
 *   log q_v = (z_v - m) / tau - l
 *   loss = sum over kept j of p_j (log p_j - log q_{id_j})    (0 where p_j = 0; one
 *                                                             below 2^-126 counts as 0)
 *   gradient dz_v = dloss / tau * (q_v - sum over kept j with id_j = v of p_j)
 * An id may occur more than once.  A row that keeps no entry, or whose kept a_j are
 * all -infinity (a padding position), has loss, m, l and gradient 0, whatever its
 * logits hold.
 *
 * Conventions are those of moe_dispatch.h, except that rows have any V and
 * stride and need only their elements' alignment.  Logits are binary16, bfloat16 or
 * fp32; a_j, the loss, m and l are fp32, and so are all sums.  Infinities and NaNs
 * propagate as the formulas say (an entry of -infinity has q = 0).
 */
#ifndef MOE_DISTILL_H
#define MOE_DISTILL_H

#include <stddef.h>
#include <stdint.h>

#include "moe_dispatch.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of scratch memory that moe_distill_forward needs (0 where it needs none:
 * ws may be NULL then; 0 for an unsupported shape). */
size_t moe_distill_workspace_bytes(int32_t T, int32_t V, int32_t dtype);

/* loss fp32 [T] and stats fp32 [T][2] = (m, l) of logits z [T][V] (dtype; row
 * stride ldz >= V, in elements); ids int32 [T][k] and teacher fp32 [T][k].
 * Supported: 1 <= k <= 1024, 1 <= V <= 2^24, T up to 2^20, 2^-64 <= tau <= 2^64, rows
 * and strides up to 2^36 elements of z in all. */
int moe_distill_forward(const void* z, int32_t dtype, int64_t ldz, int32_t T, int32_t V, const int32_t* ids,
                        const float* teacher, int32_t k, float tau, float* loss, float* stats, void* ws,
                        size_t ws_bytes, void* stream);

/* dz [T][V] (row stride lddz >= V) for the gradient dloss fp32 [T] of the loss; stats
 * from the forward call.  dz may be z itself with lddz == ldz; otherwise its rows share
 * no memory with z's (MOE_E_INVAL); rows of one stride may lie between each other, of two
 * strides not.  Elements of dz's rows past V are left as they were. */
int moe_distill_backward(const void* z, int32_t dtype, int64_t ldz, int32_t T, int32_t V, const int32_t* ids,
                         const float* teacher, int32_t k, float tau, const float* stats, const float* dloss,
                         void* dz, int64_t lddz, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_DISTILL_H */
