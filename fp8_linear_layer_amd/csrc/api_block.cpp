// C-ABI front end of a gated block's operators (te_block.h): argument validation, dispatch, per-call logging.  The
// rules are those of api.cpp: every check runs on the host before anything is enqueued, nothing is allocated, nothing
// synchronises.
#include <cmath>
#include <cstdio>

#include "api_checks.h"
#include "block_internal.h"
#include "te_block.h"

namespace {

constexpr int64_t kMaxK = (int64_t)1 << 22;
constexpr int64_t kMaxRowBytes = (int64_t)1 << 26;   // (64 rows of a wave within 32 bits)
constexpr int64_t kMaxDropoutCols = (int64_t)1 << 31;

tefp8::Fmt fmt_of(te_dtype_t d) { return d == TE_DTYPE_E5M2 ? tefp8::FMT_E5M2 : tefp8::FMT_E4M3; }

te_status_t check_gated(const char* fn, const void* a, const float* a_scales, te_dtype_t a_dtype, const void* b, const float* b_scales,
                        te_dtype_t b_dtype, int64_t M, int64_t H, int64_t K, te_activation_t act, te_accum_t accum)
{
    if (M < 1 || M >= kMaxRows) return report(TE_ERR_INVALID_ARGUMENT, "%s: M must be in [1, 2^31) (got %lld)", fn, (long long)M);
    if (H < 128 || H % 128 != 0 || H > kMaxK)
        return report(TE_ERR_INVALID_ARGUMENT, "%s: H must be a positive multiple of 128 up to 2^22 (got %lld)", fn, (long long)H);
    if (K < 128 || K % 128 != 0 || K > kMaxK)
        return report(TE_ERR_INVALID_ARGUMENT, "%s: K must be a positive multiple of 128 up to 2^22 (got %lld)", fn, (long long)K);
    if (act != TE_ACT_SILU && act != TE_ACT_GELU) return report(TE_ERR_INVALID_ARGUMENT, "%s: activation %d is none", fn, (int)act);
    if (accum != TE_ACCUM_FULL_FP32 && accum != TE_ACCUM_FAST)
        return report(TE_ERR_INVALID_ARGUMENT, "%s: accumulation policy %d is none", fn, (int)accum);
    if (!is_fp8(a_dtype) || !is_fp8(b_dtype))
        return report(TE_ERR_INVALID_ARGUMENT, "%s: operands must be TE_DTYPE_E4M3 or TE_DTYPE_E5M2 (got %d, %d)", fn, (int)a_dtype,
                      (int)b_dtype);
    TE_CHECK(check_array(fn, "the first operand", a, 16));
    TE_CHECK(check_array(fn, "the first operand's scales", a_scales, 16));
    TE_CHECK(check_array(fn, "the weight", b, 16));
    TE_CHECK(check_array(fn, "the weight's scales", b_scales, 16));
    return TE_OK;
}

// The result [M][cols] (cols a multiple of 128), plain or in fp8 in one or both layouts.
te_status_t check_result(const char* fn, const void* out, te_dtype_t dtype, int64_t ld, uint32_t flags, const float* scales, const void* qt,
                         int64_t ld_qt, const float* scales_t, int64_t M, int64_t cols)
{
    const bool fp8 = is_fp8(dtype);
    if (!fp8 && !is_float(dtype)) return report(TE_ERR_INVALID_ARGUMENT, "%s: output type %d is no type", fn, (int)dtype);
    if (flags & ~(uint32_t)(fp8 ? TE_CAST_POW2_SCALE : 0))
        return report(TE_ERR_INVALID_ARGUMENT, "%s: unknown cast flag bits 0x%x", fn, flags);
    if (!fp8) {
        if (scales || qt || scales_t) return report(TE_ERR_INVALID_ARGUMENT, "%s: scales, qt and scales_t belong to fp8 outputs", fn);
        TE_CHECK(check_array(fn, "the output", out, 16));
        if (ld < cols) return report(TE_ERR_INVALID_ARGUMENT, "%s: the output's row stride is below its row length", fn);
        if (ld % (dtype == TE_DTYPE_BF16 ? 8 : 4) != 0)
            return report(TE_ERR_MISALIGNED, "%s: the output's rows must be 16-byte aligned", fn);
        if (ld * size_of(dtype) >= kMaxRowBytes) return report(TE_ERR_UNSUPPORTED, "%s: the output's row stride is 64 MiB or more", fn);
        return TE_OK;
    }
    if ((out == nullptr) != (scales == nullptr) || (qt == nullptr) != (scales_t == nullptr) || (!out && !qt))
        return report(TE_ERR_INVALID_ARGUMENT, "%s: codes with scales, qt with scales_t, at least one of the two", fn);
    if (out) {
        if (ld < cols) return report(TE_ERR_INVALID_ARGUMENT, "%s: the codes' row stride is below their row length", fn);
        if (!aligned(out, 16) || ld % 16 != 0 || !aligned(scales, 16))
            return report(TE_ERR_MISALIGNED, "%s: codes, their row stride and scales must be 16-byte aligned", fn);
        if (ld >= kMaxRowBytes) return report(TE_ERR_UNSUPPORTED, "%s: the codes' row stride is 64 MiB or more", fn);
    }
    if (qt) {
        if (M % 128 != 0)
            return report(TE_ERR_INVALID_ARGUMENT, "%s: the cast of the transpose needs M to be a multiple of 128 (got %lld)", fn, (long long)M);
        if (ld_qt < M) return report(TE_ERR_INVALID_ARGUMENT, "%s: ld_qt must be >= M", fn);
        if (!aligned(qt, 16) || ld_qt % 16 != 0 || !aligned(scales_t, 16))
            return report(TE_ERR_MISALIGNED, "%s: qt, its row stride and scales_t must be 16-byte aligned", fn);
    }
    return TE_OK;
}

te_status_t check_z(const char* fn, const void* z, int64_t ld, int64_t H)
{
    TE_CHECK(check_array(fn, "z", z, 16));
    if (ld < 2 * H) return report(TE_ERR_INVALID_ARGUMENT, "%s: z's row stride must be >= 2 H", fn);
    if (ld % 8 != 0) return report(TE_ERR_MISALIGNED, "%s: z's rows must be 16-byte aligned", fn);
    if (ld >= kMaxRowBytes / 2) return report(TE_ERR_UNSUPPORTED, "%s: z's row stride is 64 MiB or more", fn);
    return TE_OK;
}

tefp8::GemmArgs gated_args(const void* a, const float* sa, te_dtype_t fa, const void* b, const float* sb, te_dtype_t fb, int64_t M, int64_t N,
                           int64_t K, te_activation_t act, te_accum_t accum)
{
    tefp8::GemmArgs g{};
    g.a = static_cast<const uint8_t*>(a);
    g.sa = sa;
    g.b = static_cast<const uint8_t*>(b);
    g.sb = sb;
    g.M = M;
    g.N = N;
    g.lda = g.ldb = K;
    g.lsa = te_scale_ld(M);
    g.lsb = te_scale_ld(N);
    g.fmt_a = fmt_of(fa);
    g.fmt_b = fmt_of(fb);
    g.fast = accum == TE_ACCUM_FAST;
    g.flags = (uint32_t)act;
    g.num_groups = 1;
    g.groups[0] = tefp8::Group{0, (int32_t)(K / 128), 0, 0};
    return g;
}

void set_casts(tefp8::GemmArgs& g, void* q, te_dtype_t dtype, int64_t ld, uint32_t flags, float* scales, void* qt, int64_t ld_qt,
               float* scales_t, int64_t cols)
{
    g.q_out = static_cast<uint8_t*>(q);
    g.q_scales = scales;
    g.ld_q = ld;
    g.ld_qs = te_scale_ld(g.M);
    g.q_fmt = fmt_of(dtype);
    g.q_pow2 = (flags & TE_CAST_POW2_SCALE) != 0;
    g.qt_out = static_cast<uint8_t*>(qt);
    g.qt_scales = scales_t;
    g.ld_qt = ld_qt;
    g.ld_qts = te_scale_ld(cols);
}

te_status_t check_drop(const char* fn, float p, const int64_t* rng, tefp8::Drop& d)
{
    if (!(p >= 0.0f && p <= 1.0f)) return report(TE_ERR_INVALID_ARGUMENT, "%s: p must be in [0, 1]", fn);
    if (p > 0.0f) TE_CHECK(check_array(fn, "rng", rng, 8));
    const uint32_t drop = (uint32_t)std::floor((double)p * 65536.0 + 0.5);   // of 65536
    d.rng = rng;
    d.all = drop == 65536;
    d.below = d.all ? 0x10000u : drop << 16;
    d.factor = d.all ? 0.0f : (float)(65536.0 / (65536.0 - drop));
    return TE_OK;
}

}  // namespace

extern "C" {

int64_t te_fp8_gated_fwd_workspace_bytes(int64_t M, int64_t H, int64_t K, te_dtype_t y_dtype)
{
    if (M < 1 || H < 128 || K < 128) return 0;
    if (M <= tefp8::kFewRows) return tefp8::gated_few_workspace_bytes(M, 2 * H, is_fp8(y_dtype));
    return is_fp8(y_dtype) && tefp8::gated_fwd_through_f32(M, H) ? M * H * 4 : 0;
}

te_status_t te_fp8_gated_fwd(const void* x, const float* x_scales, te_dtype_t x_dtype, const void* w, const float* w_scales,
                             te_dtype_t w_dtype, int64_t M, int64_t H, int64_t K, te_activation_t activation, void* y, te_dtype_t y_dtype,
                             int64_t ld_y, uint32_t cast_flags, float* scales, void* qt, int64_t ld_qt, float* scales_t, void* z_bf16,
                             int64_t ld_z, void* workspace, int64_t workspace_bytes, te_accum_t accum, hipStream_t stream)
{
    const char* fn = "te_fp8_gated_fwd";
    try {
        TE_CHECK(check_gated(fn, x, x_scales, x_dtype, w, w_scales, w_dtype, M, H, K, activation, accum));
        TE_CHECK(check_result(fn, y, y_dtype, ld_y, cast_flags, scales, qt, ld_qt, scales_t, M, H));
        if (z_bf16) TE_CHECK(check_z(fn, z_bf16, ld_z, H));
        const bool fp8 = is_fp8(y_dtype);
        const bool few = M <= tefp8::kFewRows;
        const bool through = !few && fp8 && !qt && tefp8::gated_fwd_through_f32(M, H);
        if (few || !qt) TE_CHECK(check_workspace(fn, workspace, workspace_bytes, te_fp8_gated_fwd_workspace_bytes(M, H, K, y_dtype)));
        tefp8::GemmArgs g = gated_args(x, x_scales, x_dtype, w, w_scales, w_dtype, M, 2 * H, K, activation, accum);
        g.aux = static_cast<uint16_t*>(z_bf16);
        g.ld_aux = ld_z;
        if (through) {
            g.out = workspace;
            g.ld_out = H;
        } else if (fp8) {
            set_casts(g, y, y_dtype, ld_y, cast_flags, scales, qt, ld_qt, scales_t, H);
        } else {
            g.out = y;
            g.out_bf16 = y_dtype == TE_DTYPE_BF16;
            g.ld_out = ld_y;
        }
        hipError_t e = few ? tefp8::launch_gated_few(g, K, workspace, stream) : tefp8::launch_gated_fwd(g, stream);
        if (e == hipSuccess && through)
            e = tefp8::launch_cast_f32_rows(static_cast<const float*>(workspace), M, H, H, fmt_of(y_dtype),
                                            (cast_flags & TE_CAST_POW2_SCALE) != 0, static_cast<uint8_t*>(y), ld_y, scales,
                                            te_scale_ld(M), stream);
        if (tefp8::log_calls())
            std::fprintf(stderr, "[te_fp8] %s M=%lld H=%lld K=%lld x=%d w=%d y=%d act=%d accum=%d flags=0x%x transpose=%d z=%d few=%d through=%d\n",
                         fn, (long long)M, (long long)H, (long long)K, (int)x_dtype, (int)w_dtype, (int)y_dtype, (int)activation,
                         (int)accum, cast_flags, qt ? 1 : 0, z_bf16 ? 1 : 0, few ? 1 : 0, through ? 1 : 0);
        return launched(fn, e);
    } catch (...) {
        return report(TE_ERR_INTERNAL, "te_fp8_gated_fwd: internal error");
    }
}

te_status_t te_fp8_gated_dgrad(const void* dy, const float* dy_scales, te_dtype_t dy_dtype, const void* wt, const float* wt_scales,
                               te_dtype_t wt_dtype, int64_t M, int64_t H, int64_t K, te_activation_t activation, const void* z_bf16,
                               int64_t ld_z, void* dz, te_dtype_t dz_dtype, int64_t ld_dz, uint32_t cast_flags, float* scales, void* qt,
                               int64_t ld_qt, float* scales_t, te_accum_t accum, hipStream_t stream)
{
    const char* fn = "te_fp8_gated_dgrad";
    try {
        TE_CHECK(check_gated(fn, dy, dy_scales, dy_dtype, wt, wt_scales, wt_dtype, M, H, K, activation, accum));
        TE_CHECK(check_z(fn, z_bf16, ld_z, H));
        TE_CHECK(check_result(fn, dz, dz_dtype, ld_dz, cast_flags, scales, qt, ld_qt, scales_t, M, 2 * H));
        tefp8::GemmArgs g = gated_args(dy, dy_scales, dy_dtype, wt, wt_scales, wt_dtype, M, H, K, activation, accum);
        g.preact = static_cast<const uint16_t*>(z_bf16);
        g.ld_aux = ld_z;
        if (is_fp8(dz_dtype)) {
            set_casts(g, dz, dz_dtype, ld_dz, cast_flags, scales, qt, ld_qt, scales_t, 2 * H);
        } else {
            g.out = dz;
            g.out_bf16 = dz_dtype == TE_DTYPE_BF16;
            g.ld_out = ld_dz;
        }
        const hipError_t e = tefp8::launch_gated_dgrad(g, stream);
        if (tefp8::log_calls())
            std::fprintf(stderr, "[te_fp8] %s M=%lld H=%lld K=%lld dy=%d wt=%d dz=%d act=%d flags=0x%x transpose=%d\n", fn, (long long)M,
                         (long long)H, (long long)K, (int)dy_dtype, (int)wt_dtype, (int)dz_dtype, (int)activation, cast_flags, qt ? 1 : 0);
        return launched(fn, e);
    } catch (...) {
        return report(TE_ERR_INTERNAL, "te_fp8_gated_dgrad: internal error");
    }
}

te_status_t te_dropout(const void* x, te_dtype_t x_dtype, int64_t ld_x, const void* residual, te_dtype_t residual_dtype, int64_t ld_residual,
                       int64_t rows, int64_t cols, float p, const int64_t* rng, void* out, te_dtype_t out_dtype, int64_t ld_out,
                       hipStream_t stream)
{
    const char* fn = "te_dropout";
    try {
        if (rows < 0 || rows >= kMaxRows)
            return report(TE_ERR_INVALID_ARGUMENT, "%s: rows must be in [0, 2^31) (got %lld)", fn, (long long)rows);
        if (cols < 1 || cols >= kMaxDropoutCols)
            return report(TE_ERR_INVALID_ARGUMENT, "%s: cols must be in [1, 2^31) (got %lld)", fn, (long long)cols);
        tefp8::DropoutArgs a{};
        TE_CHECK(check_drop(fn, p, rng, a.drop));
        if (rows == 0) return report_ok();
        TE_CHECK(check_matrix(fn, "x", x, x_dtype, ld_x, cols));
        if (residual) TE_CHECK(check_matrix(fn, "residual", residual, residual_dtype, ld_residual, cols));
        TE_CHECK(check_matrix(fn, "out", out, out_dtype, ld_out, cols));
        if ((out == x && (out_dtype != x_dtype || (rows > 1 && ld_out != ld_x))) ||
            (out == residual && (out_dtype != residual_dtype || (rows > 1 && ld_out != ld_residual))))
            return report(TE_ERR_INVALID_ARGUMENT, "%s: in place needs one type and one row stride", fn);
        a.x = x;
        a.res = residual;
        a.out = out;
        a.rows = rows;
        a.cols = cols;
        a.ld_x = ld_x;
        a.ld_res = ld_residual;
        a.ld_out = ld_out;
        a.x_bf16 = x_dtype == TE_DTYPE_BF16;
        a.res_bf16 = residual_dtype == TE_DTYPE_BF16;
        a.out_bf16 = out_dtype == TE_DTYPE_BF16;
        const hipError_t e = tefp8::launch_dropout(a, stream);
        if (tefp8::log_calls())
            std::fprintf(stderr, "[te_fp8] %s rows=%lld cols=%lld x=%d residual=%d out=%d p=%g\n", fn, (long long)rows, (long long)cols,
                         (int)x_dtype, residual ? (int)residual_dtype : 0, (int)out_dtype, (double)p);
        return launched(fn, e);
    } catch (...) {
        return report(TE_ERR_INTERNAL, "te_dropout: internal error");
    }
}

te_status_t te_layernorm_fwd(const void* x, te_dtype_t x_dtype, int64_t ld_x, const void* residual, te_dtype_t residual_dtype,
                             int64_t ld_residual, float p, const int64_t* rng, const void* gamma_bf16, const void* beta_bf16, float eps,
                             int64_t rows, int64_t cols, void* h, int64_t ld_h, float* mean, float* rstd, void* y, te_dtype_t y_dtype,
                             int64_t ld_y, uint32_t cast_flags, float* scales, void* qt, int64_t ld_qt, float* scales_t, hipStream_t stream)
{
    const char* fn = "te_layernorm_fwd";
    try {
        TE_CHECK(check_norm_dims(fn, rows, cols));
        const bool fp8 = is_fp8(y_dtype);
        if (!fp8 && !is_float(y_dtype)) return report(TE_ERR_INVALID_ARGUMENT, "%s: y_dtype %d is no type", fn, (int)y_dtype);
        if (!(eps >= 0.0f) || std::isinf(eps)) return report(TE_ERR_INVALID_ARGUMENT, "%s: eps must be finite and not negative", fn);
        if (cast_flags & ~(uint32_t)(fp8 ? TE_CAST_POW2_SCALE : 0))
            return report(TE_ERR_INVALID_ARGUMENT, "%s: unknown cast flag bits 0x%x", fn, cast_flags);
        if (!fp8 && (scales || qt || scales_t))
            return report(TE_ERR_INVALID_ARGUMENT, "%s: scales, qt and scales_t belong to fp8 outputs", fn);
        tefp8::LayerNormFwdArgs a{};
        TE_CHECK(check_drop(fn, p, rng, a.drop));
        if (rows == 0) return report_ok();
        if (a.drop.below && !residual) return report(TE_ERR_INVALID_ARGUMENT, "%s: dropout of x needs a residual", fn);
        TE_CHECK(check_matrix(fn, "x", x, x_dtype, ld_x, cols));
        TE_CHECK(check_array(fn, "gamma", gamma_bf16, 2));
        if (beta_bf16) TE_CHECK(check_array(fn, "beta", beta_bf16, 2));
        TE_CHECK(check_array(fn, "mean", mean));
        TE_CHECK(check_array(fn, "rstd", rstd));
        if (residual) {
            TE_CHECK(check_matrix(fn, "residual", residual, residual_dtype, ld_residual, cols));
            TE_CHECK(check_matrix(fn, "h", h, residual_dtype, ld_h, cols));
            TE_CHECK(check_in_place(fn, h, ld_h, residual, ld_residual, rows));
        } else if (h) {
            return report(TE_ERR_INVALID_ARGUMENT, "%s: h given without a residual", fn);
        }
        const void* src = residual ? h : x;
        const te_dtype_t src_dtype = residual ? residual_dtype : x_dtype;
        const int64_t ld_src = residual ? ld_h : ld_x;
        if (!fp8) {
            TE_CHECK(check_matrix(fn, "y", y, y_dtype, ld_y, cols));
        } else {
            if ((y == nullptr) != (scales == nullptr) || (qt == nullptr) != (scales_t == nullptr) || (!y && !qt))
                return report(TE_ERR_INVALID_ARGUMENT, "%s: y with scales, qt with scales_t, at least one of the two", fn);
            if (y) {
                if (cols % 128 != 0)
                    return report(TE_ERR_INVALID_ARGUMENT, "%s: the fp8 cast needs cols to be a multiple of 128 (got %lld)", fn,
                                  (long long)cols);
                if (ld_y < cols) return report(TE_ERR_INVALID_ARGUMENT, "%s: ld_y must be >= cols", fn);
                if (!aligned(y, 16) || ld_y % 16 != 0 || !aligned(scales, 16))
                    return report(TE_ERR_MISALIGNED, "%s: fp8 y, its row stride and scales must be 16-byte aligned", fn);
            }
            if (qt) {
                if (rows % 128 != 0 || cols % 8 != 0)
                    return report(TE_ERR_INVALID_ARGUMENT,
                                  "%s: the cast of the transpose needs rows a multiple of 128 and cols of 8 (got %lld, %lld)", fn,
                                  (long long)rows, (long long)cols);
                if (ld_qt < rows) return report(TE_ERR_INVALID_ARGUMENT, "%s: ld_qt must be >= rows", fn);
                if (!aligned(qt, 16) || ld_qt % 16 != 0 || !aligned(scales_t, 16))
                    return report(TE_ERR_MISALIGNED, "%s: qt, its row stride and scales_t must be 16-byte aligned", fn);
                if (!aligned(src, 16) || ld_src * size_of(src_dtype) % 16 != 0)
                    return report(TE_ERR_MISALIGNED, "%s: the cast of the transpose needs %s and its rows to be 16-byte aligned", fn,
                                  residual ? "h" : "x");
            }
        }
        a.x = x;
        a.res = residual;
        a.gamma = static_cast<const uint16_t*>(gamma_bf16);
        a.beta = static_cast<const uint16_t*>(beta_bf16);
        a.h = h;
        a.mean = mean;
        a.rstd = rstd;
        a.y = y;
        a.scales = scales;
        a.qt = static_cast<uint8_t*>(qt);
        a.scales_t = scales_t;
        a.src = src;
        a.rows = rows;
        a.ld_x = ld_x;
        a.ld_res = ld_residual;
        a.ld_h = ld_h;
        a.ld_y = ld_y;
        a.ld_s = te_scale_ld(rows);
        a.ld_qt = ld_qt;
        a.ld_st = te_scale_ld(cols);
        a.ld_src = ld_src;
        a.cols = (int)cols;
        a.eps = eps;
        a.x_bf16 = x_dtype == TE_DTYPE_BF16;
        a.h_bf16 = residual_dtype == TE_DTYPE_BF16;
        a.src_bf16 = src_dtype == TE_DTYPE_BF16;
        a.out = fp8 ? tefp8::NormOut::Fp8 : y_dtype == TE_DTYPE_BF16 ? tefp8::NormOut::Bf16 : tefp8::NormOut::F32;
        a.fmt = fmt_of(y_dtype);
        a.pow2 = (cast_flags & TE_CAST_POW2_SCALE) != 0;
        const hipError_t e = tefp8::launch_layernorm_fwd(a, stream);
        if (tefp8::log_calls())
            std::fprintf(stderr, "[te_fp8] %s rows=%lld cols=%lld x=%d residual=%d y=%d flags=0x%x transpose=%d p=%g\n", fn, (long long)rows,
                         (long long)cols, (int)x_dtype, residual ? (int)residual_dtype : 0, (int)y_dtype, cast_flags, qt ? 1 : 0, (double)p);
        return launched(fn, e);
    } catch (...) {
        return report(TE_ERR_INTERNAL, "te_layernorm_fwd: internal error");
    }
}

int64_t te_layernorm_bwd_workspace_bytes(int64_t rows, int64_t cols)
{
    if (rows < 1 || cols < 1) return 0;
    return tefp8::layernorm_bwd_blocks(rows, cols) * 2 * ((cols + 3) / 4 * 4) * 4;
}

te_status_t te_layernorm_bwd(const void* dy, te_dtype_t dy_dtype, int64_t ld_dy, const void* h, te_dtype_t h_dtype, int64_t ld_h,
                             const float* mean, const float* rstd, const void* gamma_bf16, int64_t rows, int64_t cols, const void* dres,
                             int64_t ld_dres, void* dh, int64_t ld_dh, float p, const int64_t* rng, void* dx, te_dtype_t dx_dtype,
                             int64_t ld_dx, float* dgamma, float* dbeta, void* workspace, int64_t workspace_bytes, hipStream_t stream)
{
    const char* fn = "te_layernorm_bwd";
    try {
        TE_CHECK(check_norm_dims(fn, rows, cols));
        tefp8::LayerNormBwdArgs a{};
        TE_CHECK(check_drop(fn, p, rng, a.drop));
        if (rows > 0) {
            TE_CHECK(check_matrix(fn, "dy", dy, dy_dtype, ld_dy, cols));
            TE_CHECK(check_matrix(fn, "h", h, h_dtype, ld_h, cols));
            TE_CHECK(check_matrix(fn, "dh", dh, h_dtype, ld_dh, cols));
            if (dres) TE_CHECK(check_matrix(fn, "dres", dres, h_dtype, ld_dres, cols));
            TE_CHECK(check_in_place(fn, dh, ld_dh, dres, ld_dres, rows));
            if ((dx != nullptr) != (p > 0.0f)) return report(TE_ERR_INVALID_ARGUMENT, "%s: dx belongs to p > 0", fn);
            if (dx) TE_CHECK(check_matrix(fn, "dx", dx, dx_dtype, ld_dx, cols));
            TE_CHECK(check_array(fn, "mean", mean));
            TE_CHECK(check_array(fn, "rstd", rstd));
            TE_CHECK(check_array(fn, "gamma", gamma_bf16, 2));
        }
        if (dgamma || dbeta) {
            if (dgamma) TE_CHECK(check_array(fn, "dgamma", dgamma));
            if (dbeta) TE_CHECK(check_array(fn, "dbeta", dbeta));
            TE_CHECK(check_workspace(fn, workspace, workspace_bytes, te_layernorm_bwd_workspace_bytes(rows, cols)));
        }
        a.dy = dy;
        a.h = h;
        a.mean = mean;
        a.rstd = rstd;
        a.gamma = static_cast<const uint16_t*>(gamma_bf16);
        a.dres = rows > 0 ? dres : nullptr;
        a.dh = dh;
        a.dx = dx;
        a.dgamma = dgamma;
        a.dbeta = dbeta;
        a.partial = dgamma || dbeta ? static_cast<float*>(workspace) : nullptr;
        a.rows = rows;
        a.blocks = tefp8::layernorm_bwd_blocks(rows, cols);
        a.ld_dy = ld_dy;
        a.ld_h = ld_h;
        a.ld_dres = ld_dres;
        a.ld_dh = ld_dh;
        a.ld_dx = ld_dx;
        a.ld_partial = (cols + 3) / 4 * 4;
        a.cols = (int)cols;
        a.dy_bf16 = dy_dtype == TE_DTYPE_BF16;
        a.h_bf16 = h_dtype == TE_DTYPE_BF16;
        a.dx_bf16 = dx_dtype == TE_DTYPE_BF16;
        const hipError_t e = tefp8::launch_layernorm_bwd(a, stream);
        if (tefp8::log_calls())
            std::fprintf(stderr, "[te_fp8] %s rows=%lld cols=%lld dy=%d h=%d dres=%d p=%g dgamma=%d dbeta=%d blocks=%lld\n", fn, (long long)rows,
                         (long long)cols, (int)dy_dtype, (int)h_dtype, dres ? 1 : 0, (double)p, dgamma ? 1 : 0, dbeta ? 1 : 0,
                         (long long)a.blocks);
        return launched(fn, e);
    } catch (...) {
        return report(TE_ERR_INTERNAL, "te_layernorm_bwd: internal error");
    }
}

}  // extern "C"
