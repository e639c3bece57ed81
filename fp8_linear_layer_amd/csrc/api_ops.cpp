// C-ABI front end of the operators around the GEMMs (te_ops.h): argument validation, dispatch,
// per-call logging.  The rules are those of api.cpp: every check runs on the host before anything
// is enqueued, nothing is allocated, nothing synchronises.
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <vector>

#include "api_checks.h"
#include "internal.h"
#include "ops_internal.h"
#include "te_ops.h"

namespace {

constexpr int64_t kMaxCount = (int64_t)1 << 36;   // elements of a gradient: a batch's chunks are counted in 32 bits

te_status_t check_router_dims(const char* fn, int64_t tokens, int64_t experts, int32_t top_k)
{
    if (tokens < 0 || tokens >= kMaxRows)
        return report(TE_ERR_INVALID_ARGUMENT, "%s: tokens must be in [0, 2^31) (got %lld)", fn, (long long)tokens);
    if (experts < 1) return report(TE_ERR_INVALID_ARGUMENT, "%s: experts must be positive (got %lld)", fn, (long long)experts);
    if (top_k < 1 || top_k > experts)
        return report(TE_ERR_INVALID_ARGUMENT, "%s: top_k must be in [1, experts] (got %d)", fn, (int)top_k);
    if (experts > tefp8::kRouterMaxExperts || top_k > tefp8::kRouterMaxTopK)
        return report(TE_ERR_UNSUPPORTED, "%s: at most %d experts and top_k %d (got %lld, %d)", fn,
                      tefp8::kRouterMaxExperts, tefp8::kRouterMaxTopK, (long long)experts, (int)top_k);
    return TE_OK;
}

}  // namespace

extern "C" {

te_status_t te_rmsnorm_fwd(const void* x, te_dtype_t x_dtype, int64_t ld_x, const void* residual,
                           te_dtype_t residual_dtype, int64_t ld_residual, const void* gamma_bf16, float eps,
                           int64_t rows, int64_t cols, void* h, int64_t ld_h, float* rstd, void* y, te_dtype_t y_dtype,
                           int64_t ld_y, uint32_t cast_flags, float* scales, void* qt, int64_t ld_qt, float* scales_t,
                           hipStream_t stream)
{
    const char* fn = "te_rmsnorm_fwd";
    try {
        TE_CHECK(check_norm_dims(fn, rows, cols));
        const bool fp8 = is_fp8(y_dtype);
        if (!fp8 && !is_float(y_dtype)) return report(TE_ERR_INVALID_ARGUMENT, "%s: y_dtype %d is no type", fn, (int)y_dtype);
        if (!(eps >= 0.0f) || std::isinf(eps)) return report(TE_ERR_INVALID_ARGUMENT, "%s: eps must be finite and not negative", fn);
        if (cast_flags & ~(uint32_t)(fp8 ? TE_CAST_POW2_SCALE : 0))
            return report(TE_ERR_INVALID_ARGUMENT, "%s: unknown cast flag bits 0x%x", fn, cast_flags);
        if (!fp8 && (scales || qt || scales_t))
            return report(TE_ERR_INVALID_ARGUMENT, "%s: scales, qt and scales_t belong to fp8 outputs", fn);
        if (rows == 0) return report_ok();
        TE_CHECK(check_matrix(fn, "x", x, x_dtype, ld_x, cols));
        TE_CHECK(check_array(fn, "gamma", gamma_bf16, 2));
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
                    return report(TE_ERR_MISALIGNED, "%s: the cast of the transpose needs %s and its rows to be 16-byte aligned",
                                  fn, residual ? "h" : "x");
            }
        }
        tefp8::NormFwdArgs a{};
        a.x = x;
        a.res = residual;
        a.gamma = static_cast<const uint16_t*>(gamma_bf16);
        a.h = h;
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
        a.fmt = y_dtype == TE_DTYPE_E5M2 ? tefp8::FMT_E5M2 : tefp8::FMT_E4M3;
        a.pow2 = (cast_flags & TE_CAST_POW2_SCALE) != 0;
        const hipError_t e = tefp8::launch_rmsnorm_fwd(a, stream);
        if (tefp8::log_calls())
            std::fprintf(stderr, "[te_fp8] %s rows=%lld cols=%lld x=%d residual=%d y=%d flags=0x%x transpose=%d\n", fn,
                         (long long)rows, (long long)cols, (int)x_dtype, residual ? (int)residual_dtype : 0, (int)y_dtype,
                         cast_flags, qt ? 1 : 0);
        return launched(fn, e);
    } catch (...) {
        return report(TE_ERR_INTERNAL, "te_rmsnorm_fwd: internal error");
    }
}

int64_t te_rmsnorm_bwd_workspace_bytes(int64_t rows, int64_t cols)
{
    if (rows < 1 || cols < 1) return 0;
    return tefp8::rmsnorm_bwd_blocks(rows, cols) * ((cols + 3) / 4 * 4) * 4;
}

te_status_t te_rmsnorm_bwd(const void* dy, te_dtype_t dy_dtype, int64_t ld_dy, const void* h, te_dtype_t h_dtype,
                           int64_t ld_h, const float* rstd, const void* gamma_bf16, int64_t rows, int64_t cols,
                           const void* dres, int64_t ld_dres, void* dh, int64_t ld_dh, float* dgamma, void* workspace,
                           int64_t workspace_bytes, hipStream_t stream)
{
    const char* fn = "te_rmsnorm_bwd";
    try {
        TE_CHECK(check_norm_dims(fn, rows, cols));
        if (rows > 0) {
            TE_CHECK(check_matrix(fn, "dy", dy, dy_dtype, ld_dy, cols));
            TE_CHECK(check_matrix(fn, "h", h, h_dtype, ld_h, cols));
            TE_CHECK(check_matrix(fn, "dh", dh, h_dtype, ld_dh, cols));
            if (dres) TE_CHECK(check_matrix(fn, "dres", dres, h_dtype, ld_dres, cols));
            TE_CHECK(check_in_place(fn, dh, ld_dh, dres, ld_dres, rows));
            TE_CHECK(check_array(fn, "rstd", rstd));
            TE_CHECK(check_array(fn, "gamma", gamma_bf16, 2));
        }
        if (dgamma) {
            TE_CHECK(check_array(fn, "dgamma", dgamma));
            TE_CHECK(check_workspace(fn, workspace, workspace_bytes, te_rmsnorm_bwd_workspace_bytes(rows, cols)));
        }
        tefp8::NormBwdArgs a{};
        a.dy = dy;
        a.h = h;
        a.rstd = rstd;
        a.gamma = static_cast<const uint16_t*>(gamma_bf16);
        a.dres = rows > 0 ? dres : nullptr;
        a.dh = dh;
        a.dgamma = dgamma;
        a.partial = dgamma ? static_cast<float*>(workspace) : nullptr;
        a.rows = rows;
        a.blocks = tefp8::rmsnorm_bwd_blocks(rows, cols);
        a.ld_dy = ld_dy;
        a.ld_h = ld_h;
        a.ld_dres = ld_dres;
        a.ld_dh = ld_dh;
        a.ld_partial = (cols + 3) / 4 * 4;
        a.cols = (int)cols;
        a.dy_bf16 = dy_dtype == TE_DTYPE_BF16;
        a.h_bf16 = h_dtype == TE_DTYPE_BF16;
        const hipError_t e = tefp8::launch_rmsnorm_bwd(a, stream);
        if (tefp8::log_calls())
            std::fprintf(stderr, "[te_fp8] %s rows=%lld cols=%lld dy=%d h=%d dres=%d dgamma=%d blocks=%lld\n", fn,
                         (long long)rows, (long long)cols, (int)dy_dtype, (int)h_dtype, dres ? 1 : 0, dgamma ? 1 : 0,
                         (long long)a.blocks);
        return launched(fn, e);
    } catch (...) {
        return report(TE_ERR_INTERNAL, "te_rmsnorm_bwd: internal error");
    }
}

int64_t te_moe_router_workspace_bytes(int64_t tokens, int64_t experts)
{
    if (tokens < 1 || experts < 1) return 0;
    return tefp8::router_fwd_workspace_bytes(tokens, experts);
}

te_status_t te_moe_router_fwd(const void* logits, te_dtype_t logits_dtype, int64_t ld_logits, int64_t tokens,
                              int64_t experts, int32_t top_k, int32_t renormalize, const uint8_t* token_mask,
                              int32_t* index, float* weight, float* lse, int32_t* counts, int32_t* routed, float* loss,
                              void* workspace, int64_t workspace_bytes, hipStream_t stream)
{
    const char* fn = "te_moe_router_fwd";
    try {
        TE_CHECK(check_router_dims(fn, tokens, experts, top_k));
        if (!is_float(logits_dtype))
            return report(TE_ERR_INVALID_ARGUMENT, "%s: logits must be TE_DTYPE_BF16 or TE_DTYPE_F32 (got %d)", fn, (int)logits_dtype);
        const bool stats = counts || routed || loss;
        if (stats) {
            TE_CHECK(check_array(fn, "counts", counts));
            TE_CHECK(check_array(fn, "routed", routed));
            TE_CHECK(check_array(fn, "loss", loss));
            TE_CHECK(check_workspace(fn, workspace, workspace_bytes, te_moe_router_workspace_bytes(tokens, experts)));
        }
        if (tokens > 0) {
            TE_CHECK(check_matrix(fn, "logits", logits, logits_dtype, ld_logits, experts));
            TE_CHECK(check_array(fn, "index", index));
            TE_CHECK(check_array(fn, "weight", weight));
            if (lse) TE_CHECK(check_array(fn, "lse", lse));
        } else if (!stats) {
            return report_ok();
        }
        tefp8::RouterArgs a{};
        a.logits = logits;
        a.mask = token_mask;
        a.tokens = tokens;
        a.ld = ld_logits;
        a.experts = (int)experts;
        a.top_k = top_k;
        a.bf16 = logits_dtype == TE_DTYPE_BF16;
        a.renorm = renormalize != 0;
        a.index = index;
        a.weight = weight;
        a.lse = lse;
        a.counts = counts;
        a.routed = routed;
        a.loss = loss;
        // (without tokens one workgroup writes the zeros)
        a.blocks = tokens > 0 ? tefp8::router_fwd_blocks(tokens, experts, stats) : 1;
        a.workspace = stats && a.blocks > 1 ? workspace : nullptr;
        const hipError_t e = tefp8::launch_router_fwd(a, stream);
        if (tefp8::log_calls())
            std::fprintf(stderr, "[te_fp8] %s tokens=%lld experts=%lld top_k=%d logits=%d renormalize=%d mask=%d loss=%d grid=%lld\n",
                         fn, (long long)tokens, (long long)experts, (int)top_k, (int)logits_dtype, a.renorm ? 1 : 0,
                         token_mask ? 1 : 0, stats ? 1 : 0, (long long)a.blocks);
        return launched(fn, e);
    } catch (...) {
        return report(TE_ERR_INTERNAL, "te_moe_router_fwd: internal error");
    }
}

te_status_t te_moe_router_bwd(const void* logits, te_dtype_t logits_dtype, int64_t ld_logits, int64_t tokens,
                              int64_t experts, int32_t top_k, int32_t renormalize, const int32_t* index,
                              const float* lse, const float* d_weight, const int32_t* counts, const int32_t* routed,
                              const float* d_loss, void* d_logits, int64_t ld_d_logits, hipStream_t stream)
{
    const char* fn = "te_moe_router_bwd";
    try {
        TE_CHECK(check_router_dims(fn, tokens, experts, top_k));
        if (!is_float(logits_dtype))
            return report(TE_ERR_INVALID_ARGUMENT, "%s: logits must be TE_DTYPE_BF16 or TE_DTYPE_F32 (got %d)", fn, (int)logits_dtype);
        if (d_loss) {
            TE_CHECK(check_array(fn, "d_loss", d_loss));
            TE_CHECK(check_array(fn, "counts", counts));
            TE_CHECK(check_array(fn, "routed", routed));
        }
        if (tokens == 0) return report_ok();
        TE_CHECK(check_matrix(fn, "logits", logits, logits_dtype, ld_logits, experts));
        TE_CHECK(check_matrix(fn, "d_logits", d_logits, logits_dtype, ld_d_logits, experts));
        TE_CHECK(check_array(fn, "index", index));
        TE_CHECK(check_array(fn, "lse", lse));
        if (d_weight) TE_CHECK(check_array(fn, "d_weight", d_weight));
        tefp8::RouterBwdArgs a{};
        a.logits = logits;
        a.tokens = tokens;
        a.ld = ld_logits;
        a.experts = (int)experts;
        a.top_k = top_k;
        a.bf16 = logits_dtype == TE_DTYPE_BF16;
        a.renorm = renormalize != 0;
        a.index = index;
        a.lse = lse;
        a.d_weight = d_weight;
        a.counts = counts;
        a.routed = routed;
        a.d_loss = d_loss;
        a.d_logits = d_logits;
        a.ld_d = ld_d_logits;
        const hipError_t e = tefp8::launch_router_bwd(a, stream);
        if (tefp8::log_calls())
            std::fprintf(stderr, "[te_fp8] %s tokens=%lld experts=%lld top_k=%d logits=%d renormalize=%d d_weight=%d d_loss=%d\n", fn,
                         (long long)tokens, (long long)experts, (int)top_k, (int)logits_dtype, a.renorm ? 1 : 0,
                         d_weight ? 1 : 0, d_loss ? 1 : 0);
        return launched(fn, e);
    } catch (...) {
        return report(TE_ERR_INTERNAL, "te_moe_router_bwd: internal error");
    }
}

int64_t te_grad_norm_workspace_bytes(int64_t n) { return n < 0 ? 0 : tefp8::clip_workspace_bytes(); }

te_status_t te_grad_norm_clip(const te_grad_tensor_t* tensors, int64_t n, float max_norm, float* norm, void* workspace,
                              int64_t workspace_bytes, hipStream_t stream)
{
    const char* fn = "te_grad_norm_clip";
    try {
        if (n < 0 || n >= kMaxRows) return report(TE_ERR_INVALID_ARGUMENT, "%s: n must be in [0, 2^31) (got %lld)", fn, (long long)n);
        if (n > 0 && !tensors) return report(TE_ERR_INVALID_ARGUMENT, "%s: tensors is null", fn);
        if (!(max_norm > 0.0f)) return report(TE_ERR_INVALID_ARGUMENT, "%s: max_norm must be positive", fn);
        TE_CHECK(check_array(fn, "norm", norm));
        TE_CHECK(check_workspace(fn, workspace, workspace_bytes, te_grad_norm_workspace_bytes(n)));
        for (int64_t i = 0; i < n; ++i) {
            const te_grad_tensor_t& t = tensors[i];
            if (t.count < 0) return report(TE_ERR_INVALID_ARGUMENT, "%s: tensor %lld has a negative count", fn, (long long)i);
            if (!is_float(t.grad_dtype) || (t.out && !is_float(t.out_dtype)))
                return report(TE_ERR_INVALID_ARGUMENT, "%s: tensor %lld must be TE_DTYPE_BF16 or TE_DTYPE_F32", fn, (long long)i);
            if (t.count == 0) continue;
            if (!t.grad) return report(TE_ERR_INVALID_ARGUMENT, "%s: tensor %lld has a null gradient", fn, (long long)i);
            if (!aligned(t.grad, size_of(t.grad_dtype)) || (t.out && !aligned(t.out, size_of(t.out_dtype))))
                return report(TE_ERR_MISALIGNED, "%s: tensor %lld is not aligned to its elements", fn, (long long)i);
            if (t.count > kMaxCount) return report(TE_ERR_UNSUPPORTED, "%s: tensor %lld has more than 2^36 elements", fn, (long long)i);
            if (t.out == t.grad && t.out_dtype != t.grad_dtype)
                return report(TE_ERR_INVALID_ARGUMENT, "%s: tensor %lld: in place needs one type", fn, (long long)i);
        }
        // The next batch of tensors from index `at` on.
        auto fill = [&](tefp8::ClipBatch& b, int64_t at) {
            b.n = 0;
            b.chunks = 0;
            for (; at < n && b.n < tefp8::kClipBatch; ++at) {
                const te_grad_tensor_t& t = tensors[at];
                if (t.count == 0) continue;
                b.t[b.n] = tefp8::ClipTensor{t.grad, t.out, t.count};
                b.first[b.n] = b.chunks;
                b.types[b.n] = (t.grad_dtype == TE_DTYPE_BF16 ? 1 : 0) | (t.out_dtype == TE_DTYPE_BF16 ? 2 : 0);
                b.chunks += (int32_t)tefp8::clip_chunks(t.count);
                ++b.n;
            }
            return at;
        };
        double* partial = static_cast<double*>(workspace);
        int64_t bytes = 0;   // (of memory that exists: far below 2^63)
        for (int64_t i = 0; i < n; ++i) bytes += tensors[i].count * size_of(tensors[i].grad_dtype);
        const bool past = bytes >= tefp8::kClipPast;
        tefp8::ClipBatch b{};
        std::vector<int64_t> starts;
        starts.reserve((size_t)(n / tefp8::kClipBatch + 1));
        int64_t slots = 0;
        for (int64_t at = 0;;) {
            starts.push_back(at);
            const int64_t next = fill(b, at);
            const hipError_t e = tefp8::launch_grad_sumsq(b, partial, slots, past, stream);
            if (e != hipSuccess) return launched(fn, e);
            slots = std::max(slots, tefp8::clip_blocks(b));
            if (next >= n) break;
            at = next;
        }
        const int64_t launches = (int64_t)starts.size();
        for (int64_t i = launches - 1; i >= 0; --i) {
            if (i < launches - 1) fill(b, starts[(size_t)i]);   // (the last one's is there)
            const hipError_t e = tefp8::launch_grad_scale(b, partial, slots, max_norm, i == launches - 1 ? norm : nullptr, past, stream);
            if (e != hipSuccess) return launched(fn, e);
        }
        if (tefp8::log_calls())
            std::fprintf(stderr, "[te_fp8] %s n=%lld max_norm=%g batches=%lld slots=%lld past=%d\n", fn, (long long)n, (double)max_norm,
                         (long long)launches, (long long)slots, past ? 1 : 0);
        return report_ok();
    } catch (...) {
        return report(TE_ERR_INTERNAL, "te_grad_norm_clip: internal error");
    }
}

}  // extern "C"
