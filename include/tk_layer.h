/*
 * tk_layer.h -- C ABI of the operators of an MoE layer around the expert's
 * activation cast (tk.h), for AMD Instinct MI355X (gfx950):
 *
 *   tk_rmsnorm_cast_fp8  residual addition + root-mean-square norm + FP8 cast
 *   tk_rmsnorm_backward  its gradient
 *   tk_route             routing: scores, balancing bias, groups, top-k, weights
 *   tk_route_backward    the gradient of the weights to the logits
 *   tk_expert_gemv_fp4   the experts' matrix-vector products, 4-bit weights
 *
 * One decode step of an MoE block in this library's calls: tk_rmsnorm_cast_fp8
 * (residual, FP8 activations and bf16 rows for the router), the router's
 * logits, tk_route, tk_expert_gemv_fp4 (gate and up projections),
 * tk_swiglu_cast_fp8, tk_expert_gemv_fp4 (down projection), tk_moe_reduce.
 * The weights are what tk_cast_fp4 writes.
 *
 * The conventions of tk.h hold here too: device pointers owned by the caller,
 * asynchronous on `stream`, nothing allocated, every precondition checked
 * before any HIP call, errors returned.  No call needs tk_init, and every call
 * may be captured into a HIP graph.  Outputs must not overlap inputs or each
 * other except where said.  n == 0 or tokens == 0 launches nothing and returns
 * TK_OK, except for tk_rmsnorm_backward, which still writes a zero dweight.
 * Results do not depend on n, tokens or the other rows (tk_rmsnorm_backward's
 * dweight, a sum over the rows, excepted), and equal calls give equal bits.
 */
#ifndef TK_LAYER_H_
#define TK_LAYER_H_

#include <stdint.h>

#include "tk.h"

#ifdef __cplusplus
extern "C" {
#endif

/* FP8 E4M3 codes with scales, as tk_swiglu_cast_fp8, tk_cast_fp8 and
 * tk_rmsnorm_cast_fp8 write them: a tk_dtype value of tk_expert_gemv_fp4's x. */
#define TK_DTYPE_FP8 2

/* Rows of tk_rmsnorm_backward's workspace. */
#define TK_RMSNORM_PARTS 256

typedef enum {
    TK_SCORE_SIGMOID = 0, /* 1 / (1 + e^-l) of each logit */
    TK_SCORE_SOFTMAX = 1  /* e^l over the token's sum of them */
} tk_scoring;

/*
 * tk_rmsnorm_cast_fp8: adds the residual, norms each row by its root mean
 * square, multiplies by the weight and casts the result to FP8 E4M3 -- one read
 * of the inputs, one write of the outputs, one launch.
 *
 *   h    = RN_t(RN(x + residual)), t the type in_dtype (h = x without residual)
 *   rstd = RN(1 / sqrt(sum h^2 / hidden + eps))   (in 64 bits, the order of the
 *          sum fixed by hidden)
 *   y    = RN(RN(h * rstd) * weight)              (fp32)
 *   codes and scales of y as tk_cast_fp8 makes them from fp32 rows.
 * A row of zeros has codes and scales of zero (UE8M0: byte 0); a NaN or an
 * infinity in a row makes every code of it NaN (0x7F or 0xFF) or, beside an
 * infinity, zero.
 *
 *  x            [n, hidden] row-major, in_dtype elements, 16-byte aligned.
 *  residual     [n, hidden], as x; NULL: none.
 *  in_dtype     TK_DTYPE_BF16 or TK_DTYPE_FP32: x, residual and residual_out.
 *  weight       fp32 [hidden], 16-byte aligned.
 *  n, hidden    0 <= n < 2^31; hidden a positive multiple of 8, at most 32768
 *               (more: TK_ERR_UNSUPPORTED).
 *  eps          >= 0 and finite.  (eps = 0 makes a row of zeros NaN.)
 *  group_size, scale_fmt   as tk_cast_fp8.
 *  residual_out [n, hidden] of in_dtype, 16-byte aligned: h, the stream the
 *               next layer adds to; may be the x or the residual buffer itself
 *               (updated in place); NULL: not written.
 *  y            bf16 [n, hidden], 16-byte aligned: y rounded once, e.g. for the
 *               router; NULL: not written.
 *  rstd         fp32 [n], 4-byte aligned: for tk_rmsnorm_backward; NULL: not
 *               written.
 *  codes, scales  as tk_cast_fp8; both NULL: only the other outputs are written
 *               (residual_out, y or rstd, at least one of them).
 */
tk_status tk_rmsnorm_cast_fp8(const void* x, const void* residual, tk_dtype in_dtype, const float* weight, int64_t n,
                              int64_t hidden, float eps, int64_t group_size, tk_scale_fmt scale_fmt,
                              void* residual_out, void* y, float* rstd, void* codes, void* scales, void* stream);

/*
 * tk_rmsnorm_backward: the gradient of tk_rmsnorm_cast_fp8's y (the cast passes
 * it on unchanged) to h, which is that of x and of the residual alike:
 *
 *   g  = dy * weight;  a = rstd * h
 *   dx = rstd * (g - a * (sum g*a / hidden)) + dresidual
 *   dweight = sum over the rows of dy * a
 * in fp32, dx rounded once to in_dtype.  The order of every sum is fixed by n
 * and hidden.
 *
 *  dy         [n, hidden] of in_dtype: the gradient of y.
 *  h          [n, hidden] of in_dtype: the forward's residual_out (its x when
 *             there was no residual).
 *  weight     fp32 [hidden];  rstd  fp32 [n], as the forward wrote it.
 *  dresidual  [n, hidden] of in_dtype: the gradient that reaches residual_out
 *             by itself (the skip connection); NULL: none.
 *  dx         [n, hidden] of in_dtype; may be the dy or the dresidual buffer.
 *  dweight    fp32 [hidden], overwritten (zeros for n == 0); NULL: not computed.
 *  workspace  fp32 [min(n, TK_RMSNORM_PARTS), hidden]: the rows' partial sums
 *             (of many rows; not touched for few); may be NULL when dweight is
 *             NULL or n == 0.
 * [n, hidden] buffers, weight, dweight and workspace 16-byte aligned, rstd
 * 4-byte.  hidden as in the forward.
 */
tk_status tk_rmsnorm_backward(const void* dy, const void* h, tk_dtype in_dtype, const float* weight,
                              const float* rstd, const void* dresidual, int64_t n, int64_t hidden, void* dx,
                              float* dweight, float* workspace, void* stream);

/*
 * tk_route: routing of tokens to experts from the router's logits.
 *
 *   s_e   the expert's score: sigmoid of its logit, or softmax over the token's
 *         logits, computed in 64 bits.
 *   key_e = RN(s_e) + bias_e in fp32 (bias 0 when NULL) when there is a bias or
 *         n_group > 1, else the logit itself (both scores grow with it).
 *   An expert whose logit is -inf, or whose key is, is masked: never chosen.
 *   n_group > 1: the experts form n_group consecutive groups; a group's value
 *         is the sum of its two largest keys (its one key when only one expert
 *         is not masked), and only the topk_group best groups' experts stay,
 *         equal values going to the smaller group index.
 *   Then k times: the largest remaining key, equal keys to the smaller index.
 *   weight = RN(scale * s_e), or, with normalise, RN(scale * s_e / sum) over the
 *         token's chosen experts, in 64 bits and without the bias (a sum of
 *         zero leaves scale * s_e).
 *   A slot for which no expert remains (masks leave fewer than k, or none) has
 *   index -1 and weight 0; tk_topk_to_pos and tk_expert_gemv_fp4 take it as
 *   absent.  A token with a NaN among its logits or keys, or with softmax a
 *   logit of +inf, gets indices 0..k-1 and NaN weights, so that it shows.
 *
 *  logits       [tokens, experts] row-major, in_dtype elements (TK_DTYPE_FP32
 *               or TK_DTYPE_BF16), aligned to the element.
 *  bias         fp32 [experts], 4-byte aligned, or NULL.  Moves the choice only.
 *  tokens       0 <= tokens < 2^31.
 *  experts      1..512;  k  1..64 (more: TK_ERR_UNSUPPORTED), at most
 *               topk_group * experts / n_group.
 *  n_group      divides experts (1: no groups), each group of 2 experts or
 *               more; topk_group in 1..n_group.
 *  normalise    0 or 1;  scale  finite.
 *  topk_idx     int32 [tokens, k], best key first;  topk_weight  fp32
 *               [tokens, k] in the same order; 4-byte aligned.
 */
tk_status tk_route(const void* logits, tk_dtype in_dtype, const float* bias, int64_t tokens, int64_t experts,
                   int64_t k, int64_t n_group, int64_t topk_group, tk_scoring scoring, int normalise, float scale,
                   int32_t* topk_idx, float* topk_weight, void* stream);

/*
 * tk_route_backward: the gradient of tk_route's weights to the logits.  The
 * choice itself has none, nor has the bias.
 *
 *   With d_j = scale * dweight_j for the chosen experts j, w_j their scores s_j,
 *   divided by their sum S when normalised:
 *   sigmoid              dlogit_j = d_j * s_j * (1 - s_j)
 *   sigmoid, normalised  dlogit_j = (d_j - sum_i d_i w_i) / S * s_j * (1 - s_j)
 *   softmax              dlogit_e = s_e * (d_e - sum_i d_i s_i) for every e, d_e
 *                        0 where e is not chosen
 *   softmax, normalised  dlogit_j = w_j * (d_j - sum_i d_i w_i), w the softmax
 *                        of the chosen logits among themselves
 *   and 0 elsewhere, in 64 bits (softmax over all experts: from fp32
 *   exponentials), rounded to fp32 and from there to in_dtype.
 *
 *  dweight      fp32 [tokens, k];  topk_idx  int32 [tokens, k], as tk_route
 *               wrote it (an entry outside 0..experts-1 is absent; a repeated
 *               one counts once, by its first slot).
 *  logits       [tokens, experts] of in_dtype, the forward's.
 *  dlogits      [tokens, experts] of in_dtype, written whole, aligned to the
 *               element.
 *  tokens, experts, k, scoring, normalise, scale   as the forward.
 */
tk_status tk_route_backward(const float* dweight, const int32_t* topk_idx, const void* logits, tk_dtype in_dtype,
                            int64_t tokens, int64_t experts, int64_t k, tk_scoring scoring, int normalise,
                            float scale, void* dlogits, void* stream);

/*
 * tk_expert_gemv_fp4: for every token t and choice j the matrix-vector product
 *
 *   out[t*k + j] = W[topk_idx[t*k + j]] x[r],   r = t*k + j when x_slots, else t
 *
 * with 4-bit weights: W[e][o][c] = codes * scale, as tk_cast_fp4 writes them
 * from bf16 or fp32 rows [experts*out_features, in_features] with a row-major
 * scale_fmt.  Products and sums in fp32, rounded once to out_dtype.  Codes with
 * UE8M0 scales enter as bf16 numbers, which hold every weight, and every
 * activation down to 2^-133: what an E4M3 code has below that under the scale
 * bytes 0, 1 and 2 is rounded away (values of 2^128 and more are infinite, as in
 * fp32).  A chosen expert's weights are read once
 * for its rows together, up to 16 at a time: made for a step of decoding, a few
 * rows an expert.
 *
 *  x            [tokens, in_features], or [tokens*k, in_features] when x_slots;
 *               TK_DTYPE_BF16 elements, or TK_DTYPE_FP8 codes with x_scales.
 *               16-byte aligned.
 *  x_scales     NULL for TK_DTYPE_BF16 (x_scale_fmt and x_group are then
 *               ignored).  For TK_DTYPE_FP8: row-major scales, x_scale_fmt
 *               TK_SCALE_FP32 or TK_SCALE_UE8M0 (other layouts:
 *               TK_ERR_UNSUPPORTED), one for each x_group columns (0: one a
 *               row).
 *  topk_idx     int32 [tokens, k], 4-byte aligned; an entry outside
 *               0..experts-1 gives a row of zeros.  NULL: every row uses expert
 *               0, and k is 1.
 *  tokens, k    tokens * k < 2^31; k  1..64 (more: TK_ERR_UNSUPPORTED).
 *  codes        uint8 [experts, out_features, in_features/2], 16-byte aligned.
 *  scales       [experts, out_features, in_features/group], scale_fmt
 *               TK_SCALE_UE8M0 or TK_SCALE_FP32 (4-byte aligned).
 *  group_size   0 (one scale a row) or a divisor of in_features: a multiple of
 *               32 for UE8M0, of 128 for FP32 (other widths that divide:
 *               TK_ERR_UNSUPPORTED); x_group likewise.
 *  experts      1..32768;  out_features  1..2^24;  in_features  a positive
 *               multiple of 32, at most 2^20.
 *  out_dtype    TK_DTYPE_BF16 or TK_DTYPE_FP32.
 *  out          [tokens*k, out_features], aligned to the element.
 */
tk_status tk_expert_gemv_fp4(const void* x, const void* x_scales, int x_dtype, tk_scale_fmt x_scale_fmt,
                             int64_t x_group, const int32_t* topk_idx, int64_t tokens, int64_t k, int x_slots,
                             const void* codes, const void* scales, tk_scale_fmt scale_fmt, int64_t group_size,
                             int64_t experts, int64_t out_features, int64_t in_features, tk_dtype out_dtype,
                             void* out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TK_LAYER_H_ */
