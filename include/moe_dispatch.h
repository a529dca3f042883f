/*
 * moe_dispatch.h -- tokens laid out by expert and back, and the gradients of
 * that path, for training what sits around the 4-bit experts of
 * moe_w4a16.h (the router, adapters) and for expert products outside it.
 *
 * With idx[t][j] the expert of token t's slot j (moe_route's topk_idx; any
 * value outside [0, E) is a dropped slot, as adaptive top-p leaves -1) and
 * w[t][j] its weight:
 *   sort       the kept slots ("pairs", id t*k + j) ordered by expert, and by
 *              pair id within an expert; each expert's group starts at a
 *              multiple of `align` rows
 *   dispatch   xs[pos(t,j)] = x[t]
 *     gradient dx[t] = sum_j dxs[pos(t,j)]
 *   combine    y[t] = sum_j w[t][j] * o[pos(t,j)]
 *     gradient do[pos(t,j)] = w[t][j] * dy[t],  dw[t][j] = <dy[t], o[pos(t,j)]>
 *   router     w_j = s_j / S, s_j = sigmoid(z_j), S = sum of the kept s_j,
 *              z_j = b[e_j] + <x[t], Wr[e_j]>
 *     gradient dz_j = w_j * (1 - s_j) * (dw_j - sum_i dw_i w_i)
 *              dx[t] = sum_j dz_j Wr[e_j],  dWr[e] = sum over e's pairs of
 *              dz * x[t],  db[e] = sum over e's pairs of dz
 *              (the choice of experts itself has no gradient).
 *
 * Conventions are those of moe_w4a16.h (device pointers, caller-owned
 * buffers, validation before any launch, nothing allocates, copies,
 * synchronises, prints or throws, every call can be captured in a HIP graph),
 * with these differences:
 *   - Rows (x, xs, o, y, dy, ...) are binary16, bfloat16 or fp32 (moe_dtype_t),
 *     H a multiple of 8, 16-byte aligned; int32 and fp32 arrays (idx, w, pos,
 *     pairs, offsets, dw, db) 4-byte aligned, router_w and its gradient 16.
 *   - Workspaces need no initial contents and 16-byte alignment; calls that
 *     overlap in time must not share one.
 *   - Sums are held in fp32 (the router's logits too, which moe_route forms
 *     in fp64) and rounded once to the rows' type.  Infinities
 *     and NaNs propagate as the formulas say; rows of dropped slots and
 *     padding rows are never read.  Bitwise the same at every call (no
 *     floating-point atomics).
 *   - Index contents are checked on the device: an entry of idx, pos, pairs or
 *     offsets outside its range is treated as dropped and nothing outside the
 *     buffers is read or written.
 *   - Shapes: 1 <= k <= E, 0 <= T, 1 <= align <= 1024, else MOE_E_INVAL;
 *     T <= 2^20, k <= 32, E <= 1024, H <= 65536, and in moe_combine_backward
 *     and moe_route_backward rows <= 2^25 + 2^20 (no sort gives more), else
 *     MOE_E_UNSUPPORTED.
 *     T == 0 launches nothing and returns MOE_OK, except where a call has an
 *     output that does not depend on T (offsets, d_o's padding rows, dWr, db),
 *     which is written.
 */
#ifndef MOE_DISPATCH_H
#define MOE_DISPATCH_H

#include <stddef.h>
#include <stdint.h>

#include "moe_w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { MOE_T_F16 = 0, MOE_T_BF16 = 1, MOE_T_F32 = 2 } moe_dtype_t;

/* Rows of the expert-sorted buffers for T tokens: T * k when align == 1;
 * otherwise T * k + min(E, T * k) * (align - 1), rounded up to a multiple of
 * align (the most that padding every group can take).  -1 for a shape
 * outside the supported set or 2^31 rows and more. */
int64_t moe_sort_rows(int32_t T, int32_t k, int32_t n_experts, int32_t align);

/* Bytes of scratch memory that moe_sort and moe_dispatch need.  0 where they
 * need none (up to 32,768 slots: ws may be NULL) and for an unsupported shape. */
size_t moe_sort_workspace_bytes(int32_t T, int32_t k, int32_t n_experts);

/* Sorts the slots of topk_idx (int32 [T][k]) by expert.
 *   offsets int32 [E + 1]: expert e's group starts at row offsets[e]; it holds
 *     its pairs and then padding up to offsets[e + 1] (a multiple of align);
 *   pairs int32 [rows]: pair id of each row, -1 for padding rows and for the
 *     rows past offsets[E];
 *   pos int32 [T][k]: row of each slot, -1 for a dropped slot. */
int moe_sort(const int32_t* topk_idx, int32_t T, int32_t k, int32_t n_experts, int32_t align, int32_t* offsets,
             int32_t* pairs, int32_t* pos, void* ws, size_t ws_bytes, void* stream);

/* moe_sort, and the rows: xs [rows][H] receives x[t] (x: [T][H]) in the row
 * of each kept slot and zeros in every other row. */
int moe_dispatch(const void* x, int32_t dtype, int32_t T, int32_t H, const int32_t* topk_idx, int32_t k,
                 int32_t n_experts, int32_t align, void* xs, int32_t* offsets, int32_t* pairs, int32_t* pos,
                 void* ws, size_t ws_bytes, void* stream);

/* dx [T][H] = add + sum_j dxs[pos(t,j)]; dxs [rows][H]; add [T][H] or NULL
 * (it may be dx itself).  A token without kept slots gets add, or zeros. */
int moe_dispatch_backward(const void* dxs, int32_t dtype, int32_t rows, int32_t H, const int32_t* pos, int32_t T,
                          int32_t k, const void* add, void* dx, void* stream);

/* y [T][H] = add + sum_j topk_w[t][j] * o[pos(t,j)]; o [rows][H]; topk_w fp32
 * [T][k]; add [T][H] or NULL (for instance the shared expert's rows; it may be
 * y itself). */
int moe_combine(const void* o, int32_t dtype, int32_t rows, int32_t H, const float* topk_w, const int32_t* pos,
                int32_t T, int32_t k, const void* add, void* y, void* stream);

/* Gradients of moe_combine for dy [T][H]: d_o [rows][H] (zeros in rows whose
 * `pairs` entry is none of the T * k slots, or a slot that pos drops), dw fp32
 * [T][k] (0 for dropped slots).  pos and pairs come from one moe_sort. */
int moe_combine_backward(const void* dy, const void* o, int32_t dtype, int32_t rows, int32_t H,
                         const float* topk_w, const int32_t* pos, const int32_t* pairs, int32_t T, int32_t k,
                         void* d_o, float* dw, void* stream);

/* Bytes of scratch memory that moe_route_backward needs (0 for an unsupported
 * shape); rows as passed to the call. */
size_t moe_route_backward_workspace_bytes(int32_t T, int32_t k, int32_t n_experts, int32_t H, int32_t rows);

/* Gradients of the router's weights (moe_route's topk_w) for dw fp32 [T][k]:
 * dx [T][H] = add + sum_j dz_j Wr[e_j] (add [T][H] or NULL, may be dx);
 * d_router_w fp32 [E][H]; d_router_b fp32 [E].
 *   x [T][H], binary16 or bfloat16; router_w fp32 [E][H]; router_b fp32 [E] or
 *   NULL; topk_idx int32 [T][k]; offsets and pairs [rows] from moe_sort of
 *   that topk_idx (any align). */
int moe_route_backward(const void* x, int32_t dtype, int32_t T, int32_t H, int32_t n_experts, int32_t k,
                       const float* router_w, const float* router_b, const int32_t* topk_idx, const float* dw,
                       const int32_t* offsets, const int32_t* pairs, int32_t rows, const void* add, void* dx,
                       float* d_router_w, float* d_router_b, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_DISPATCH_H */
