/*
 * tk_expert.h -- C ABI of the experts' matrix products of a prefill and of
 * training, for AMD Instinct MI355X (gfx950):
 *
 *   tk_expert_gemm            out = x W^T, rows grouped by expert
 *   tk_expert_gemm_dgrad      its gradient to the rows, dx = dy W
 *   tk_expert_gemm_wgrad      its gradient to the weights, dW = dy^T x, from
 *                             bf16 rows or their FP8 checkpoint
 *   tk_swiglu_checkpoint_fp8  SwiGLU + cast, which also leaves its input in FP8
 *   tk_swiglu_backward        the gradient of SwiGLU, from that checkpoint
 *
 * Rows are laid out as tk_topk_to_pos (tk.h) makes them: expert 0's first, then
 * expert 1's, ..., expert_offsets on the device.  A training step of an expert
 * block: tk_cast_fp8 or tk_rmsnorm_cast_fp8 (x in FP8, kept for the backward
 * pass), tk_expert_gemm (gate and up), tk_swiglu_checkpoint_fp8 (activation and
 * checkpoint), tk_expert_gemm (down), tk_moe_reduce; backward:
 * tk_expert_gemm_dgrad and _wgrad (down), tk_swiglu_backward,
 * tk_expert_gemm_dgrad and _wgrad (gate and up), tk_moe_reduce with weights 1.
 * A prefill of a block that decodes through tk_expert_gemv_fp4: tk_expert_gemm
 * with the same 4-bit weights.
 *
 * The conventions of tk.h hold here too: device pointers owned by the caller,
 * asynchronous on `stream`, nothing allocated, every precondition checked
 * before any HIP call, errors returned.  Every call is one launch and may be
 * captured into a HIP graph (tk_swiglu_checkpoint_fp8: after tk_init).  Outputs
 * must not overlap inputs or each other except where said.  Equal calls give
 * equal bits; there are no atomics on results.
 *
 * Rows of the products.  expert_offsets is int32 [experts + 1]: expert e has the
 * rows expert_offsets[e] .. expert_offsets[e + 1] - 1 of n_rows.  Entries below 0
 * or above n_rows count as these, an entry below the one before it as an expert
 * without rows (where that gives a row to two experts, the results of the call are
 * unspecified, and nothing but its outputs is written); NULL: one expert (experts is 1) has all n_rows.  Rows that no
 * expert has, such as those from expert_offsets[experts] on, are not read and
 * their results are left as they were.  n_rows may thus be a capacity: tokens*k.
 * A row index is int32 [n_rows]: the row of x (or dy) that each row takes, e.g.
 * its token, with the number of those rows given; an entry outside 0 .. rows-1
 * stands for a row of zeros, whose products with the weights are zeros whatever
 * the weights hold (in the weights' gradient, times an infinity or a NaN in the
 * other operand's row, a NaN as with any zero).  NULL: each row its own (the
 * number of rows is then n_rows or more).  Products of more tiles than one launch
 * holds (2^23 of 256 x 256 results, or 2^24 of the smallest, 64 x 16):
 * TK_ERR_UNSUPPORTED.  The tiles are chosen by n_rows / experts, since how the rows
 * lie is not known on the host: rows that nearly all fall to a few of many experts
 * are multiplied in smaller tiles, and more slowly, than those would choose alone.
 */
#ifndef TK_EXPERT_H_
#define TK_EXPERT_H_

#include <stdint.h>

#include "tk.h"
#include "tk_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* FP4 E2M1 codes with scales, as tk_cast_fp4 writes them: a tk_dtype value of
 * tk_expert_gemm's w. */
#define TK_DTYPE_FP4 3

/*
 * tk_expert_gemm: out[r] = W[e] x[i] for every row r of every expert e, i its
 * index (or r).
 *
 * bf16 x bf16: products exact, sums in fp32, one running sum over the whole
 * depth (fp32 results of normal numbers are off by some 6e-9 sqrt(depth) of
 * their norm; so are both gradients').  FP8 x FP8 and FP8 x FP4 on the matrix
 * instruction for them, 128 columns at a time: sums in fp32, but of each 128
 * products what lies some 2^-14 below the largest is dropped, which a bf16
 * result does not show as long as the sum is not much smaller than its largest
 * term; so they have no fp32 results, and a sum that nearly cancels differs from
 * that of tk_expert_gemv_fp4, whose products are exact.  UE8M0 scales of groups
 * of columns enter the instruction, one scale a row is applied to the finished
 * sum, and fp32 scales of groups to each 128 columns' sum, all in fp32: a sum
 * with its groups' scales, and the product of two fp32 scales of groups, have to
 * lie in its range; of two scales a row only their product and the result have
 * to.  A scale that is a NaN (UE8M0 byte 255) makes one of what it scales.
 *
 *  x            [x_rows, in_features]: TK_DTYPE_BF16 elements, or TK_DTYPE_FP8
 *               codes with x_scales.  16-byte aligned.
 *  x_scales     for FP8: row-major TK_SCALE_FP32 or TK_SCALE_UE8M0 (other
 *               layouts: TK_ERR_UNSUPPORTED), one for each x_group columns (0:
 *               one a row): a divisor of in_features that is a multiple of 32
 *               (UE8M0) or 128 (FP32) columns (other divisors:
 *               TK_ERR_UNSUPPORTED).  For bf16 NULL, x_scale_fmt and x_group
 *               then being ignored.
 *  x_rows       0 <= x_rows < 2^31; with 0, x and x_scales may be NULL (an empty
 *               tensor has no address), as dy may be with 0 dy_rows.
 *  row_index    int32 [n_rows], 4-byte aligned, or NULL.
 *  expert_offsets  int32 [experts + 1], 4-byte aligned, or NULL (experts 1).
 *  n_rows       0 <= n_rows < 2^31.
 *  w            [experts, out_features, in_features]: TK_DTYPE_BF16 elements (x
 *               bf16), TK_DTYPE_FP8 or TK_DTYPE_FP4 codes (x FP8; other pairs:
 *               TK_ERR_UNSUPPORTED) as tk_cast_fp8 or tk_cast_fp4 write them
 *               from rows [experts*out_features, in_features].  16-byte aligned.
 *  w_scales, w_scale_fmt, w_group  as those of x, [experts, out_features, ..].
 *  experts      1..512 (more: TK_ERR_UNSUPPORTED).
 *  out_features, in_features  positive multiples of 8 (in_features of 32 for FP8
 *               x), at most 2^20.
 *  out_dtype    TK_DTYPE_BF16, or TK_DTYPE_FP32 for bf16 operands (else
 *               TK_ERR_UNSUPPORTED).
 *  out          [n_rows, out_features], 16-byte aligned.
 */
tk_status tk_expert_gemm(const void* x, const void* x_scales, int x_dtype, tk_scale_fmt x_scale_fmt, int64_t x_group,
                         int64_t x_rows, const int32_t* row_index, const int32_t* expert_offsets, int64_t n_rows,
                         const void* w, const void* w_scales, int w_dtype, tk_scale_fmt w_scale_fmt, int64_t w_group,
                         int64_t experts, int64_t out_features, int64_t in_features, tk_dtype out_dtype, void* out,
                         void* stream);

/*
 * tk_expert_gemm_dgrad: dx[r] = W[e]^T dy[i], bf16 operands, products exact, sums
 * in fp32, rounded once to out_dtype.
 *
 *  dy         bf16 [dy_rows, out_features], 16-byte aligned.
 *  row_index  the row of dy for each row (the gradient of a sum over a token's
 *             rows is the same for all of them), or NULL.
 *  w          bf16 [experts, out_features, in_features], 16-byte aligned.
 *  out_dtype  TK_DTYPE_BF16 or TK_DTYPE_FP32: dx.
 *  dx         [n_rows, in_features], 16-byte aligned.
 * The rest as tk_expert_gemm.
 */
tk_status tk_expert_gemm_dgrad(const void* dy, int64_t dy_rows, const int32_t* row_index,
                               const int32_t* expert_offsets, int64_t n_rows, const void* w, int64_t experts,
                               int64_t out_features, int64_t in_features, tk_dtype out_dtype, void* dx, void* stream);

/*
 * tk_expert_gemm_wgrad: dW[e][o][c] = sum over e's rows r of dy[i][o] * x[j][c],
 * i and j the row's indices, sums in fp32 in the rows' order, rounded once to
 * out_dtype.
 *
 *  dy          bf16 [dy_rows, out_features], 16-byte aligned.
 *  dy_index, x_index  int32 [n_rows] or NULL.
 *  x           [x_rows, in_features]: TK_DTYPE_BF16, or TK_DTYPE_FP8 codes, with
 *              which x_scales are row-major UE8M0 bytes, one for each x_group
 *              columns (0: one a row; else a divisor of in_features that is a
 *              multiple of 8; other divisors: TK_ERR_UNSUPPORTED).  Their values,
 *              code * 2^(byte-127), are bf16 numbers, so that the products are
 *              exact (those of fp32 scales would not be); below 2^-133 they are
 *              rounded, from 2^128 on infinite, and under the byte 255 NaN.
 *  accumulate  0: dw is overwritten, with zeros for an expert without rows; 1:
 *              the sum is added to dw in fp32 before the rounding.
 *  dw          [experts, out_features, in_features] of out_dtype (TK_DTYPE_BF16
 *              or TK_DTYPE_FP32), 16-byte aligned.
 * The rest as tk_expert_gemm (in_features a multiple of 16 for FP8 x).  n_rows ==
 * 0 still writes zeros unless accumulate.
 */
tk_status tk_expert_gemm_wgrad(const void* dy, int64_t dy_rows, const int32_t* dy_index, const void* x,
                               const void* x_scales, int x_dtype, int64_t x_group, int64_t x_rows,
                               const int32_t* x_index, const int32_t* expert_offsets, int64_t n_rows, int64_t experts,
                               int64_t out_features, int64_t in_features, int accumulate, tk_dtype out_dtype, void* dw,
                               void* stream);

/*
 * tk_swiglu_checkpoint_fp8: tk_swiglu_cast_fp8(x, ..., codes, scales) and
 * tk_cast_fp8(x as [n, 2*hidden] bf16 rows, ..., x_codes, x_scales) in one read
 * of x, with the bits of those two calls.  x_codes and x_scales are the
 * checkpoint that tk_swiglu_backward takes.
 *
 *  x, topk_weight, n, hidden, clamp_limit  as tk_swiglu_cast_fp8 (no counter).
 *  group_size   of the activation's columns and of x's alike: 8, 16, 32, 64, 128,
 *               256 or 512, dividing hidden (other valid widths:
 *               TK_ERR_UNSUPPORTED, the two calls have them).
 *  scale_fmt    TK_SCALE_FP32 or TK_SCALE_UE8M0, row-major, for both (other
 *               layouts: TK_ERR_UNSUPPORTED).
 *  codes        uint8 [n, hidden], 8-byte aligned;  scales  [n, hidden/group].
 *  x_codes      uint8 [n, 2*hidden], 8-byte aligned;  x_scales  [n,
 *               2*hidden/group].
 */
tk_status tk_swiglu_checkpoint_fp8(const void* x, const float* topk_weight, int64_t n, int64_t hidden,
                                   int64_t group_size, float clamp_limit, tk_scale_fmt scale_fmt, void* codes,
                                   void* scales, void* x_codes, void* x_scales, void* stream);

/*
 * tk_swiglu_backward: the gradient of y = silu(g) * u * weight to g, u and the
 * weight, from the packed g | u as bf16 or as its FP8 checkpoint, and y itself
 * again, for the weight gradient of the product after it.
 *
 *   With the clamp L: g' = min(g, L), u' = min(max(u, -L), L); without: g, u.
 *   s = 1 / (1 + e^-g'), a = g' s
 *   dg = dy * weight * u' * (s + a * (1 - s))   where g <= L, else 0
 *   du = dy * weight * a                        where |u| <= L, else 0
 *   dweight = sum over the columns of dy * a * u'
 *   y = a * u' * weight
 * in fp32, rounded once to the outputs' types.  The sum's order is fixed by
 * hidden.  (The checkpoint's own rounding is not undone: the gradient is that at
 * the values it holds.)
 *
 *  dy           bf16 [n, hidden], 16-byte aligned.
 *  h            [n, 2*hidden], 16-byte aligned: TK_DTYPE_BF16 elements, or
 *               TK_DTYPE_FP8 codes with h_scales.
 *  h_scales     for FP8: row-major, scale_fmt TK_SCALE_FP32 (4-byte aligned) or
 *               TK_SCALE_UE8M0 (other layouts: TK_ERR_UNSUPPORTED), one for each
 *               group_size columns of 2*hidden (0: one a row; else a multiple of
 *               8 that divides 2*hidden).  For bf16 NULL, scale_fmt and
 *               group_size then being ignored.
 *  topk_weight  fp32 [n], 4-byte aligned; NULL: weight 1.
 *  n, hidden    0 <= n < 2^31; hidden a positive multiple of 8, at most 2^18.
 *  clamp_limit  L > 0; +INFINITY: no clamp.
 *  dh           bf16 [n, 2*hidden], 16-byte aligned; may be h itself when that is
 *               bf16.
 *  dweight      fp32 [n], 4-byte aligned; NULL: not computed.
 *  y            bf16 [n, hidden], 16-byte aligned; may be dy itself; NULL: not
 *               written.
 */
tk_status tk_swiglu_backward(const void* dy, const void* h, const void* h_scales, int h_dtype, tk_scale_fmt scale_fmt,
                             int64_t group_size, const float* topk_weight, int64_t n, int64_t hidden,
                             float clamp_limit, void* dh, float* dweight, void* y, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TK_EXPERT_H_ */
