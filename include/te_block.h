/*
 * te_block.h - C ABI of the operators of a gated transformer block (same
 * library, same conventions as te_fp8.h and te_ops.h):
 *
 *   te_fp8_gated_fwd, te_fp8_gated_dgrad   gated feed-forward product: both
 *                                          projections, the activation and the
 *                                          product in one GEMM, and the data
 *                                          gradient of the next GEMM through it
 *   te_layernorm_fwd, te_layernorm_bwd     layer norm with the dropped branch's and
 *                                          the residual's addition, stored in bf16 /
 *                                          fp32 or as the next GEMM's fp8 operand
 *   te_dropout                             dropout (and its gradient), with the
 *                                          residual's addition
 *
 * Device pointers owned by the caller, nothing allocated, no synchronisation,
 * arguments validated on the host before anything is enqueued, errors as
 * te_status_t with te_last_error_message().  Every call can be captured into a
 * HIP graph, and every result is the same from run to run (no floating-point
 * atomics).  Calls that may run at the same time need workspaces of their own.
 *
 * bf16 and fp32 matrices of the norm and of dropout need only the alignment of
 * their elements, and any row stride >= the row's length.  A matrix without
 * rows is accepted there and its pointers may be null.
 */
#ifndef TE_BLOCK_H
#define TE_BLOCK_H

#include "te_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* 0 is deliberately no activation: a zero-initialised argument is rejected. */
typedef enum {
    TE_ACT_SILU = 1, /* act(g) = g / (1 + exp(-g)) */
    TE_ACT_GELU = 2  /* GELU, tanh form, as TE_EPI_GELU */
} te_activation_t;

/*
 * Forward of a gated feed-forward layer:
 *   z = x * w^T                       [M][2H], fp32 accumulation
 *   y = act(gate) * up                [M][H], from the unrounded projections
 * The gate's and the up projection's features alternate in blocks of 16: rows
 * 32 b .. 32 b + 15 of w, and those columns of z, are gate features 16 b ..
 * 16 b + 15, the next 16 are the same features of up.  (Both projections of a
 * feature then meet in one lane of the matrix cores' output.)
 *
 * y is stored, by y_dtype,
 *   TE_DTYPE_BF16 / TE_DTYPE_F32   as y [M][ld_y];
 *   TE_DTYPE_E4M3 / TE_DTYPE_E5M2  as the per-token cast of the fp32 y
 *       (te_cast_fp8_per_token: 1x128 groups, scales [H/128][te_scale_ld(M)])
 *       in y and scales, and / or as the cast of its transpose (groups of 128
 *       rows; M a multiple of 128) in qt [H][ld_qt] and scales_t
 *       [M/128][te_scale_ld(H)].  Either pair may be null, not both.  A group
 *       that holds what is NaN or infinite gets a NaN scale (its codes are
 *       unspecified).
 *
 *  x, x_scales   [M][K] fp8, [K/128][te_scale_ld(M)] fp32
 *  w, w_scales   [2H][K] fp8, [K/128][te_scale_ld(2H)] fp32
 *  M >= 1;  H, K >= 128, multiples of 128 (H is the contraction length of the
 *                product that reads y); both at most 2^22
 *  z_bf16        [M][ld_z] bf16, the rounded projections for the backward
 *                pass, ld_z >= 2H, or null
 *  ld_y          % 8 == 0 for bf16, % 4 for fp32, % 16 for fp8; ld_z % 8 == 0;
 *                row strides of y and z are below 64 MiB
 *  workspace     16-byte aligned, te_fp8_gated_fwd_workspace_bytes(...) bytes
 *                (contents irrelevant; unused with qt above 128 rows)
 *  accum         as in te_fp8_gemm_fwd (TE_ACCUM_FAST chains the blocks of e4m3
 *                operands on power-of-two scales; other formats take FULL's
 *                update).  Up to 128 rows both policies sum the
 *                products of a block exactly but for fp32 roundings (a kernel of
 *                their own, on bf16 copies of the codes); otherwise with the
 *                precision of the matrix cores' fp8 sums (about 1.5e-5 of the
 *                terms' size, as in the GEMMs of te_fp8.h).  FAST's power-of-two test is
 *                taken per tile of the kernel that runs, and the outputs that are
 *                asked for choose that kernel: on scales of which only some are
 *                powers of two, results may differ between such calls within
 *                that precision.  Under FULL they do not.
 */
int64_t te_fp8_gated_fwd_workspace_bytes(int64_t M, int64_t H, int64_t K, te_dtype_t y_dtype);
te_status_t te_fp8_gated_fwd(const void* x, const float* x_scales, te_dtype_t x_dtype,
                             const void* w, const float* w_scales, te_dtype_t w_dtype,
                             int64_t M, int64_t H, int64_t K, te_activation_t activation,
                             void* y, te_dtype_t y_dtype, int64_t ld_y, uint32_t cast_flags, float* scales,
                             void* qt, int64_t ld_qt, float* scales_t,
                             void* z_bf16, int64_t ld_z, void* workspace, int64_t workspace_bytes,
                             te_accum_t accum, hipStream_t stream);

/*
 * Its backward pass, in the data gradient of the GEMM that read y:
 *   D    = dy * wt^T                  [M][H] (wt = W2^T, cast along out)
 *   dz   = (D * up * act'(gate), D * act(gate))   [M][2H], z's order of columns
 * stored as te_fp8_gated_fwd stores y (dz [M][ld_dz]; fp8 scales
 * [2H/128][te_scale_ld(M)]; qt [2H][ld_qt], scales_t [M/128][te_scale_ld(2H)]):
 * dx = dz W and dW = dz^T x follow with te_fp8_gemm_dgrad and
 * te_fp8_wgrad_accum.
 *
 *  dy, dy_scales [M][K] fp8, [K/128][te_scale_ld(M)] fp32
 *  wt, wt_scales [H][K] fp8, [K/128][te_scale_ld(H)] fp32
 *  z_bf16        [M][ld_z] bf16, the forward's
 *  accum         both policies run TE_ACCUM_FULL_FP32's update, at every M with
 *                the precision of the matrix cores' fp8 sums
 */
te_status_t te_fp8_gated_dgrad(const void* dy, const float* dy_scales, te_dtype_t dy_dtype,
                               const void* wt, const float* wt_scales, te_dtype_t wt_dtype,
                               int64_t M, int64_t H, int64_t K, te_activation_t activation,
                               const void* z_bf16, int64_t ld_z,
                               void* dz, te_dtype_t dz_dtype, int64_t ld_dz, uint32_t cast_flags, float* scales,
                               void* qt, int64_t ld_qt, float* scales_t,
                               te_accum_t accum, hipStream_t stream);

/*
 * Dropout of a matrix of `cols` columns: element (row, col) is kept if
 *   bits(row, col) >= round(p * 65536),
 * where bits are 16 of the 128 that Philox 4x32 with 10 rounds (Salmon et al.,
 * "Parallel random numbers: as easy as 1, 2, 3", 2011) gives for the key
 * rng[0] and the counter (col / 8, row, low and high half of rng[1]): word
 * (col % 8) / 2, its low half for an even column.  Kept elements are
 * multiplied by 65536 / (65536 - round(p * 65536)), dropped ones are 0 whatever
 * they were.  So p takes effect as a multiple of 2^-16; p = 1 drops all.  The
 * mask is a function of rng, row and column only and never stored: the same
 * rng in the backward pass gives the same mask.
 *
 *  rng           two 64-bit numbers in device memory, read by the kernels: the
 *                seed, and a number that differs from call to call
 */

/*
 * out = dropout(x) + residual (fp32, rounded to out's type); without a residual
 * out = dropout(x), which is also its gradient's form: dx = dropout(dy).
 *
 *  x, residual, out   TE_DTYPE_BF16 or TE_DTYPE_F32, each on its own
 *  rows, cols    rows in [0, 2^31), cols in [1, 2^31)
 *  out           may be x's or the residual's own buffer (same type and stride)
 *  p             in [0, 1]; rng as above (null only with p = 0)
 */
te_status_t te_dropout(const void* x, te_dtype_t x_dtype, int64_t ld_x,
                       const void* residual, te_dtype_t residual_dtype, int64_t ld_residual,
                       int64_t rows, int64_t cols, float p, const int64_t* rng,
                       void* out, te_dtype_t out_dtype, int64_t ld_out, hipStream_t stream);

/*
 * Layer norm:
 *   h    = dropout(x) + residual, rounded to the residual's type and stored
 *          (h = x without a residual; h's pointer must then be null, and p 0)
 *   mean = mean over the row of h;  rstd = 1 / sqrt(mean of (h - mean)^2 + eps)
 *   y    = ((h - mean) * rstd) * gamma + beta                    (all fp32)
 * stored by y_dtype as te_rmsnorm_fwd stores its y: bf16 / fp32, or fp8 in
 * either or both layouts (cols a multiple of 128 for the row-wise cast, rows
 * of 128 and cols of 8 for the transposed), NaN scales for groups that hold what
 * is not finite.
 *
 *  x, residual   TE_DTYPE_BF16 or TE_DTYPE_F32, each on its own
 *  gamma, beta   [cols] bf16; beta may be null (0)
 *  cols          1 .. 32768
 *  h             may be the residual's own buffer (the sum in place; same stride)
 *  mean, rstd    [rows] fp32, for the backward pass
 *  p, rng        dropout of x as te_dropout's; p = 0: none (rng may be null)
 */
te_status_t te_layernorm_fwd(const void* x, te_dtype_t x_dtype, int64_t ld_x,
                             const void* residual, te_dtype_t residual_dtype, int64_t ld_residual,
                             float p, const int64_t* rng, const void* gamma_bf16, const void* beta_bf16, float eps,
                             int64_t rows, int64_t cols, void* h, int64_t ld_h, float* mean, float* rstd,
                             void* y, te_dtype_t y_dtype, int64_t ld_y, uint32_t cast_flags, float* scales,
                             void* qt, int64_t ld_qt, float* scales_t, hipStream_t stream);

/*
 * Its gradient, with xh = (h - mean) * rstd and g = dy * gamma (fp32):
 *   dh     = rstd * (g - mean of g - xh * mean of g * xh) + dres   (row means)
 *   dx     = dropout(dh), from the unrounded dh
 *   dgamma = sum over the rows of dy * xh,  dbeta = sum over the rows of dy
 * dh is the gradient of the residual, dx that of x (without dropout dh is the
 * gradient of both, and dx must be null).
 *
 *  dy            TE_DTYPE_BF16 or TE_DTYPE_F32
 *  h             what the norm was of: the stored h, or x without a residual
 *  dres          the gradient that reaches h from elsewhere, h's type, or null
 *  dh            h's type; may be dres's own buffer (same stride)
 *  dx            TE_DTYPE_BF16 or TE_DTYPE_F32, needed with p > 0 (never with 0)
 *  dgamma, dbeta [cols] fp32, overwritten; null: not computed
 *  workspace     16-byte aligned, te_layernorm_bwd_workspace_bytes(rows, cols)
 *                bytes (contents irrelevant; unused without dgamma and dbeta)
 */
int64_t te_layernorm_bwd_workspace_bytes(int64_t rows, int64_t cols);
te_status_t te_layernorm_bwd(const void* dy, te_dtype_t dy_dtype, int64_t ld_dy,
                             const void* h, te_dtype_t h_dtype, int64_t ld_h, const float* mean, const float* rstd,
                             const void* gamma_bf16, int64_t rows, int64_t cols,
                             const void* dres, int64_t ld_dres, void* dh, int64_t ld_dh,
                             float p, const int64_t* rng, void* dx, te_dtype_t dx_dtype, int64_t ld_dx,
                             float* dgamma, float* dbeta, void* workspace, int64_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TE_BLOCK_H */
