/*
 * moe_adapter.h -- low-rank adapters of many requests at once beside a shared
 * projection (the 4-bit layer of moe_w4a16.h, one of its experts, or any
 * other product whose rows are passed as `add`), for serving and training.
 *
 * Adapter a has A_a [R][K], B_a [N][R], a scale s_a and a rank r_a <= R; row t
 * uses adapter ids[t] (any value outside [0, n): none).
 *   forward   u[t] = A_a x[t],  y[t] = add[t] + s_a * B_a u[t]
 *   backward  v[t] = s_a * B_a^T dy[t],  dx[t] = add[t] + A_a^T v[t]
 *             dA_a = sum_t v[t] x[t]^T,  dB_a = s_a * sum_t dy[t] u[t]^T
 * with the sums over the rows of the adapter.  Rows of A_a and columns of B_a
 * at or past r_a are not used, and their gradients are zero.
 *
 * Conventions are those of moe_dispatch.h.  Rows and adapters are binary16 or
 * bfloat16 (one moe_dtype_t for all); products of theirs are exact, sums, u and v
 * among them, are held in fp32, outputs are rounded once.  As factors in their
 * turn u and v count to 22 bits in binary16 (no finer than 2^-38 of the largest of
 * the row, or in d_a and d_b of the adapter's rows), and in bfloat16 to 16 bits in y
 * and dx and to 24 in d_a and d_b.  An infinity in any operand, or a product past
 * fp32's range, gives the infinity or NaN of the formula.  x, dy, y, dx and add may
 * have rows of a wider buffer (ld: elements from row to row, a multiple of 8).
 */
#ifndef MOE_ADAPTER_H
#define MOE_ADAPTER_H

#include <stddef.h>
#include <stdint.h>

#include "moe_dispatch.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A set of adapters (host struct holding device pointers).  Supported: K and N
 * multiples of 8 up to 65536, R a multiple of 8 up to 128, 1 <= n <= 1024, at
 * most 2^20 rows and 2^35 elements of x or dy. */
typedef struct {
  const void* a;        /* [n][R][K]                                     */
  const void* b;        /* [n][N][R]                                     */
  const float* scale;   /* fp32 [n]                                      */
  const int32_t* ranks; /* int32 [n] (values clamped to [0, R]), or NULL: all R */
  int32_t n, K, N, R;
  int32_t dtype;        /* MOE_T_F16 or MOE_T_BF16                        */
} moe_adapters_t;

/* Bytes of scratch memory that a forward / backward call on T rows needs (0
 * for an unsupported shape). */
size_t moe_adapter_workspace_bytes(const moe_adapters_t* d, int32_t T);

/* y [T][N] = add + s_a B_a (A_a x).
 *   x [T][K] with row stride ldx; ids int32 [T]; add [T][N] with row stride
 *   ldadd, or NULL (it may be y itself: the projection's rows updated in
 *   place); y with row stride ldy;
 *   u: fp32 [T][R] or NULL, receives A_a x (zeros past the rank and for rows
 *   without an adapter), which the backward call takes;
 *   offsets, pairs: moe_sort of ids as [T][1] with n experts and align 1, or
 *   both NULL: the call groups the rows itself (a caller with several
 *   projections per step sorts once and passes the result to each).  (Of a row
 *   with an adapter that they do not name, y, u and dx are not written.) */
int moe_adapter_forward(const moe_adapters_t* d, const void* x, int64_t ldx, int32_t T, const int32_t* ids,
                        const int32_t* offsets, const int32_t* pairs, const void* add, int64_t ldadd, void* y,
                        int64_t ldy, float* u, void* ws, size_t ws_bytes, void* stream);

/* Gradients for dy [T][N] (row stride lddy): dx [T][K] (row stride lddx) =
 * add + A_a^T v, or dx NULL to skip it; d_a fp32 [n][R][K] and d_b fp32
 * [n][N][R], written whole (zeros for adapters without rows).  x, ids,
 * offsets and pairs as in the forward call, u its output. */
int moe_adapter_backward(const moe_adapters_t* d, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                         const float* u, int32_t T, const int32_t* ids, const int32_t* offsets,
                         const int32_t* pairs, const void* add, int64_t ldadd, void* dx, int64_t lddx, float* d_a,
                         float* d_b, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_ADAPTER_H */
