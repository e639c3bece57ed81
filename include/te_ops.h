/*
 * te_ops.h - C ABI of the operators that stand around the FP8 GEMMs in a
 * transformer block's step (same library, same conventions as te_fp8.h):
 *
 *   te_rmsnorm_fwd, te_rmsnorm_bwd   root-mean-square norm with the residual's
 *                                    addition, stored in bf16 / fp32 or as the next
 *                                    GEMM's fp8 operand (and the weight gradient's)
 *   te_moe_router_fwd, _bwd          top-k router with per-expert counts and a
 *                                    balance loss (the counts size the grouped GEMMs)
 *   te_grad_norm_clip                global norm of many gradients, and clipping
 *
 * As in te_fp8.h: device pointers owned by the caller, nothing allocated, no
 * synchronisation, arguments validated on the host before anything is
 * enqueued, errors as te_status_t with te_last_error_message().  Every call can
 * be captured into a HIP graph, and every result is the same from run to run
 * (no floating-point atomics).
 *
 * bf16 and fp32 matrices need only the alignment of their elements, and any
 * row stride >= the row's length; fp8 outputs, and what the cast of the
 * transpose reads, need 16 bytes (pointers and row strides).  A matrix without
 * rows (or tokens) is accepted and its pointers may be null.
 */
#ifndef TE_OPS_H
#define TE_OPS_H

#include "te_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Root-mean-square norm:
 *   v    = x + residual, rounded to the residual's type and stored as h
 *          (v = x when residual is null; h must then be null too)
 *   rstd = 1 / sqrt(mean over the row of v^2 + eps)               (fp32)
 *   y    = (v * rstd) * gamma                                     (fp32)
 * and y is stored, by y_dtype,
 *   TE_DTYPE_BF16 / TE_DTYPE_F32   as y [rows][ld_y];
 *   TE_DTYPE_E4M3 / TE_DTYPE_E5M2  as the per-token cast of the fp32 y (as
 *       te_cast_fp8_per_token defines it: 1x128 groups, scales block-major
 *       [cols/128][te_scale_ld(rows)]; cols a multiple of 128) in y and scales,
 *       and / or as the cast of its transpose (groups of 128 rows, rows a
 *       multiple of 128, cols a multiple of 8) in qt [cols][ld_qt] and scales_t
 *       [rows/128][te_scale_ld(cols)].  Either pair may be null, not both.
 *       Non-finite values: where a group of either cast holds a y that is NaN
 *       or infinite, its scale is NaN, so all that the group stands for is (its
 *       codes are unspecified).
 *
 *  x, residual   TE_DTYPE_BF16 or TE_DTYPE_F32, each on its own
 *  gamma         [cols] bf16
 *  cols          1 .. 32768
 *  h             may be the residual's own buffer (the sum in place; same stride)
 *  rstd          [rows] fp32, for the backward pass
 *  cast_flags    0 or TE_CAST_POW2_SCALE
 */
te_status_t te_rmsnorm_fwd(const void* x, te_dtype_t x_dtype, int64_t ld_x,
                           const void* residual, te_dtype_t residual_dtype, int64_t ld_residual,
                           const void* gamma_bf16, float eps, int64_t rows, int64_t cols,
                           void* h, int64_t ld_h, float* rstd,
                           void* y, te_dtype_t y_dtype, int64_t ld_y, uint32_t cast_flags, float* scales,
                           void* qt, int64_t ld_qt, float* scales_t, hipStream_t stream);

/*
 * Its gradient, with xh = h * rstd and g = dy * gamma (fp32):
 *   dh     = rstd * (g - xh * mean over the row of g * xh) + dres
 *   dgamma = sum over the rows of dy * xh
 * dh is the gradient of x and of the residual alike.
 *
 *  dy            TE_DTYPE_BF16 or TE_DTYPE_F32
 *  h             what the norm was of: the stored h, or x without a residual
 *  dres          the gradient that reaches h from elsewhere, h's type, or null
 *  dh            h's type; may be dres's own buffer (same stride)
 *  dgamma        [cols] fp32, overwritten; null: not computed
 *  workspace     16-byte aligned, te_rmsnorm_bwd_workspace_bytes(rows, cols)
 *                bytes (contents irrelevant; unused without dgamma)
 */
int64_t te_rmsnorm_bwd_workspace_bytes(int64_t rows, int64_t cols);
te_status_t te_rmsnorm_bwd(const void* dy, te_dtype_t dy_dtype, int64_t ld_dy,
                           const void* h, te_dtype_t h_dtype, int64_t ld_h, const float* rstd,
                           const void* gamma_bf16, int64_t rows, int64_t cols,
                           const void* dres, int64_t ld_dres, void* dh, int64_t ld_dh, float* dgamma,
                           void* workspace, int64_t workspace_bytes, hipStream_t stream);

/*
 * Top-k router.  With p = softmax of a token's logits, the token goes to the
 * top_k experts of the largest logits, equal ones by the lower index.  A logit
 * of -inf closes its expert to the token; where fewer than top_k are open, and
 * in every entry of a masked token, index is -1 and weight 0.  A NaN logit is
 * never chosen, and makes the token's lse and weights NaN (and the loss).
 *   weight = p of the chosen experts (renormalize: divided by their sum)
 *   lse    = log of the sum of exp(logits), 0 for a token that goes nowhere
 *   counts[e] = tokens sent to expert e;  routed = n, tokens sent anywhere
 *   loss   = experts / (top_k n^2) * sum over e of
 *            counts[e] * (sum over the routed tokens of p[token][e])
 *
 *  logits        [tokens][ld] TE_DTYPE_BF16 or TE_DTYPE_F32
 *  experts       1 .. 2048;  top_k 1 .. min(16, experts)
 *  token_mask    [tokens] bytes, 0 = not routed; null: all are
 *  index, weight [tokens][top_k] int32, fp32
 *  lse           [tokens] fp32, or null
 *  counts, routed, loss   [experts] int32, [1] int32, [1] fp32, or all null
 *  workspace     16-byte aligned, te_moe_router_workspace_bytes(tokens, experts)
 *                bytes (contents irrelevant; unused without counts)
 */
int64_t te_moe_router_workspace_bytes(int64_t tokens, int64_t experts);
te_status_t te_moe_router_fwd(const void* logits, te_dtype_t logits_dtype, int64_t ld_logits, int64_t tokens,
                              int64_t experts, int32_t top_k, int32_t renormalize, const uint8_t* token_mask,
                              int32_t* index, float* weight, float* lse, int32_t* counts, int32_t* routed,
                              float* loss, void* workspace, int64_t workspace_bytes, hipStream_t stream);

/*
 * Its gradient with respect to the logits, for given gradients of the weights
 * and of the loss (the choice of experts, counts and n are constants):
 *   a[e] = d_loss * experts / (top_k n^2) * counts[e]
 *   weights p:      b = a + d_weight at the chosen e;  d = p * (b - sum of p b)
 *   renormalize:    d = p * (a - sum of p a)
 *                       + w * (d_weight - sum of w d_weight) at the chosen e
 * Tokens that went nowhere get zeros.
 *
 *  index, lse, counts, routed   the forward call's (counts, routed and d_loss
 *                all null: no loss); the indices of a token differ
 *  d_weight      [tokens][top_k] fp32, or null; ignored where index is -1
 *  d_loss        [1] fp32 in device memory
 *  d_logits      [tokens][ld_d_logits], the logits' type
 */
te_status_t te_moe_router_bwd(const void* logits, te_dtype_t logits_dtype, int64_t ld_logits, int64_t tokens,
                              int64_t experts, int32_t top_k, int32_t renormalize, const int32_t* index,
                              const float* lse, const float* d_weight, const int32_t* counts, const int32_t* routed,
                              const float* d_loss, void* d_logits, int64_t ld_d_logits, hipStream_t stream);

/*
 * Global gradient norm and clipping:
 *   norm = sqrt(sum over all tensors of g^2)          (fp64 sums, stored as fp32)
 *   out  = g * min(1, max_norm / (norm + 1e-6))       (rounded to out's type)
 * A norm that is NaN makes every output NaN; one that is infinite makes the
 * finite gradients zero.
 *
 *  tensors       host array of n descriptors, read during the call; each tensor
 *                has `count` elements (at most 2^36) one after the other, aligned
 *                to an element.  out may be grad itself (same type: in place, and not
 *                touched where the coefficient is 1, as it is for a norm of at most
 *                max_norm - 1e-6) or null (only its part of the norm); apart from
 *                that no output overlaps a gradient or another output
 *  max_norm      > 0
 *  norm          [1] fp32
 *  workspace     16-byte aligned, te_grad_norm_workspace_bytes(n) bytes
 */
typedef struct {
    const void* grad;
    void* out;
    int64_t count;
    te_dtype_t grad_dtype, out_dtype; /* TE_DTYPE_BF16 or TE_DTYPE_F32 */
} te_grad_tensor_t;

int64_t te_grad_norm_workspace_bytes(int64_t n);
te_status_t te_grad_norm_clip(const te_grad_tensor_t* tensors, int64_t n, float max_norm, float* norm,
                              void* workspace, int64_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TE_OPS_H */
