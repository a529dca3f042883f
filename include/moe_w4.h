/*
 * moe_w4.h -- products of rows with frozen 4-bit weights that have a scale per
 * group of columns: a projection or an output head beside the layer of
 * moe_w4a16.h (n = 1), or the matrices of n experts applied to rows laid out
 * by moe_dispatch; and the gradient of the rows.
 *
 *   W_e[r][c] = (q_e[r][c] - z_e[r][c / group]) * s_e[r][c / group]
 *   forward   y[t] = add[t] + W_e x[t]         for the rows t of expert e
 *   backward  dx[t] = add[t] + W_e^T dy[t]
 * The rows of expert e are offsets[e] .. offsets[e + 1] - 1; rows outside every
 * group get add[t], or zeros.  Without offsets (n = 1) all rows are used.
 *
 * Conventions are those of moe_dispatch.h.  Rows and scales are binary16 or
 * bfloat16 (one moe_dtype_t for all), codes int4 two's complement, zero points
 * int8.  Sums are fp32 and rounded once.  In forward calls of few rows
 * (moe_w4_few_rows) the codes q - z are exact factors and a group's sum is multiplied
 * by its scale in fp32.  Otherwise, and in all backward calls, the weight (q - z) s is
 * rounded to the rows' type before it is multiplied, as a 16-bit model's weights are
 * (binary16: to no finer than 2^-24, and infinite from 65520 on).  Scales are finite;
 * where weights are rounded, bfloat16 scales are at most 2^117 in magnitude.
 * Infinities and NaNs in rows propagate as the formulas say; rows of other experts and
 * rows outside the groups are never read.  A row's values do not depend on the rows
 * beside it where calls have the same T and n.
 */
#ifndef MOE_W4_H
#define MOE_W4_H

#include <stddef.h>
#include <stdint.h>

#include "moe_dispatch.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Shape of n matrices of N rows and K columns (host struct).  Supported: K a
 * multiple of 32 up to 65536, N a multiple of 8 up to 2^20, 1 <= n <= 1024, n * N
 * at most 2^24; group 32, 64, a multiple of 128, or K, and a divisor of K; zeros 0
 * (no zero points: z = 0) or 1; dtype MOE_T_F16 or MOE_T_BF16. */
typedef struct {
  int32_t n, N, K, group, zeros, dtype;
} moe_w4_dims_t;

/* Bytes of the n packed matrices (0 for an unsupported shape). */
size_t moe_w4_packed_bytes(const moe_w4_dims_t* d);

/* Canonical weights -> packed device layout, once when they are loaded:
 *   q uint8 [n][N][K / 2], column 2j in the low nibble of byte j; scales [n][N][K /
 *   group]; zeros int8 [n][N][K / group], NULL iff d->zeros == 0; packed: 256-byte
 *   aligned.  Values are unchanged. */
int moe_w4_pack(const moe_w4_dims_t* d, const void* q, const void* scales, const void* zeros, void* packed,
                void* stream);

/* Inverse of moe_w4_pack. */
int moe_w4_unpack(const moe_w4_dims_t* d, const void* packed, void* q, void* scales, void* zeros, void* stream);

/* 1 if a forward call on T rows takes the path for few rows (see above). */
int32_t moe_w4_few_rows(const moe_w4_dims_t* d, int32_t T);

/* Bytes of scratch memory that a forward (backward == 0) or backward call on T rows
 * needs (0 for an unsupported shape, and where a call needs none: ws may be NULL then). */
size_t moe_w4_workspace_bytes(const moe_w4_dims_t* d, int32_t T, int32_t backward);

/* y [T][N] (row stride ldy) = add + W_e x; x [T][K] (row stride ldx); add [T][N]
 * (row stride ldadd) or NULL (it may be y itself).  Otherwise y's rows share no memory
 * with x's or add's (MOE_E_INVAL); rows of one stride may lie between each other, of two
 * strides not.  offsets int32 [n + 1], ascending, as moe_sort gives them (any align),
 * or NULL if n == 1.  Row strides are multiples of 8 up to 2^22; T up to 2^20, and at
 * most 2^35 elements of x or y.  (Offsets are clamped to 0 .. T; where they descend, y
 * is unspecified.) */
int moe_w4_forward(const moe_w4_dims_t* d, const void* packed, const void* x, int64_t ldx, int32_t T,
                   const int32_t* offsets, const void* add, int64_t ldadd, void* y, int64_t ldy, void* ws,
                   size_t ws_bytes, void* stream);

/* dx [T][K] (row stride lddx) = add + W_e^T dy; dy [T][N] (row stride lddy);
 * add [T][K] or NULL (it may be dx itself).  Otherwise as the forward call. */
int moe_w4_backward(const moe_w4_dims_t* d, const void* packed, const void* dy, int64_t lddy, int32_t T,
                    const int32_t* offsets, const void* add, int64_t ldadd, void* dx, int64_t lddx, void* ws,
                    size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_W4_H */
