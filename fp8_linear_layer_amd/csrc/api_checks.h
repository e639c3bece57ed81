// Argument checks shared by the operators' C-ABI front ends (api_ops.cpp, api_block.cpp).
#pragma once

#include <cstdint>

#include "ops_internal.h"
#include "te_fp8.h"

namespace {

using tefp8::report;
using tefp8::report_ok;

constexpr int64_t kMaxRows = (int64_t)1 << 31;

[[maybe_unused]] bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
[[maybe_unused]] bool is_fp8(te_dtype_t d) { return d == TE_DTYPE_E4M3 || d == TE_DTYPE_E5M2; }
[[maybe_unused]] bool is_float(te_dtype_t d) { return d == TE_DTYPE_BF16 || d == TE_DTYPE_F32; }
[[maybe_unused]] int size_of(te_dtype_t d) { return d == TE_DTYPE_F32 ? 4 : d == TE_DTYPE_BF16 ? 2 : 1; }

// A bf16 or fp32 matrix [..][ld] of rows of `cols` elements.
[[maybe_unused]] te_status_t check_matrix(const char* fn, const char* what, const void* p, te_dtype_t d, int64_t ld, int64_t cols)
{
    if (!p) return report(TE_ERR_INVALID_ARGUMENT, "%s: %s pointer is null", fn, what);
    if (!is_float(d))
        return report(TE_ERR_INVALID_ARGUMENT, "%s: %s must be TE_DTYPE_BF16 or TE_DTYPE_F32 (got %d)", fn, what, (int)d);
    if (ld < cols)
        return report(TE_ERR_INVALID_ARGUMENT, "%s: row stride of %s (%lld) is below its row length %lld", fn, what,
                      (long long)ld, (long long)cols);
    if (!aligned(p, size_of(d))) return report(TE_ERR_MISALIGNED, "%s: %s is not aligned to its elements", fn, what);
    return TE_OK;
}

// An output [..][ld] that may be an input's own buffer: at another row stride its rows would be written over rows that
// are still to be read.
[[maybe_unused]] te_status_t check_in_place(const char* fn, const void* out, int64_t ld, const void* in, int64_t ld_in, int64_t rows)
{
    if (in && out == in && rows > 1 && ld != ld_in)
        return report(TE_ERR_INVALID_ARGUMENT, "%s: in place needs one row stride (got %lld, %lld)", fn, (long long)ld, (long long)ld_in);
    return TE_OK;
}

[[maybe_unused]] te_status_t check_array(const char* fn, const char* what, const void* p, int align = 4)
{
    if (!p) return report(TE_ERR_INVALID_ARGUMENT, "%s: %s pointer is null", fn, what);
    if (!aligned(p, align)) return report(TE_ERR_MISALIGNED, "%s: %s must be %d-byte aligned", fn, what, align);
    return TE_OK;
}

[[maybe_unused]] te_status_t check_workspace(const char* fn, const void* ws, int64_t have, int64_t need)
{
    if (need <= 0) return TE_OK;
    if (!ws) return report(TE_ERR_INVALID_ARGUMENT, "%s: workspace is null", fn);
    if (have < need)
        return report(TE_ERR_INVALID_ARGUMENT, "%s: workspace has %lld bytes, %lld are needed", fn, (long long)have,
                      (long long)need);
    if (!aligned(ws, 16)) return report(TE_ERR_MISALIGNED, "%s: workspace must be 16-byte aligned", fn);
    return TE_OK;
}

[[maybe_unused]] te_status_t launched(const char* fn, hipError_t e)
{
    if (e != hipSuccess) return report(TE_ERR_HIP, "%s: kernel launch failed: %s", fn, hipGetErrorString(e));
    return report_ok();
}

[[maybe_unused]] te_status_t check_norm_dims(const char* fn, int64_t rows, int64_t cols)
{
    if (rows < 0 || rows >= kMaxRows)
        return report(TE_ERR_INVALID_ARGUMENT, "%s: rows must be in [0, 2^31) (got %lld)", fn, (long long)rows);
    if (cols < 1) return report(TE_ERR_INVALID_ARGUMENT, "%s: cols must be positive (got %lld)", fn, (long long)cols);
    if (cols > tefp8::kNormMaxCols)
        return report(TE_ERR_UNSUPPORTED, "%s: cols is at most %d (got %lld)", fn, tefp8::kNormMaxCols, (long long)cols);
    return TE_OK;
}

#define TE_CHECK(call)                        \
    do {                                      \
        const te_status_t st_ = (call);       \
        if (st_ != TE_OK) return st_;         \
    } while (0)

}  // namespace
