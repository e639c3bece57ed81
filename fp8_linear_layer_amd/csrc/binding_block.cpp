// The Python side of a gated block's operators (te_block.h): checks what the C ABI cannot see of a tensor, allocates
// the outputs that are not given, and calls the C function, as binding.cpp does for te_ops.h.
#include <limits>

#include "binding_util.h"
#include "te_block.h"

namespace {

struct Library {
    decltype(&te_fp8_gated_fwd) gated_fwd;
    decltype(&te_fp8_gated_fwd_workspace_bytes) gated_fwd_workspace_bytes;
    decltype(&te_fp8_gated_dgrad) gated_dgrad;
    decltype(&te_layernorm_fwd) layernorm_fwd;
    decltype(&te_layernorm_bwd) layernorm_bwd;
    decltype(&te_layernorm_bwd_workspace_bytes) layernorm_bwd_workspace_bytes;
    decltype(&te_dropout) dropout;
    decltype(&te_status_string) status_string;
    decltype(&te_last_error_message) last_error_message;
} lib{};

bool is_fp8(int64_t type) { return type == TE_DTYPE_E4M3 || type == TE_DTYPE_E5M2; }

// An fp8 operand: codes [rows][k] and scales [k/128][rows rounded up to a multiple of 4], both contiguous.
void operand(const at::Tensor& q, const at::Tensor& scales, const char* name, const at::Device& device)
{
    if (q.device() != device || !q.is_cuda() || q.dim() != 2) refuse("%s: expected a matrix on the GPU", name);
    if (q.element_size() != 1) refuse("%s: expected fp8 codes (got %s)", name, c10::toString(q.scalar_type()));
    if (!q.is_contiguous()) refuse("%s: expected a contiguous matrix", name);
    if (q.size(1) % 128) refuse("%s: columns must be a multiple of 128 (got %lld)", name, (long long)q.size(1));
    const std::string what = std::string(name) + "_scales";
    array(scales, what.c_str(), kF32, {q.size(1) / 128, (q.size(0) + 3) / 4 * 4}, device);
}

// The generator's state where there is dropout.
const int64_t* state(const at::Tensor& rng, double p, const at::Device& device)
{
    if (!(p >= 0.0 && p <= 1.0)) refuse("p must be in [0, 1]");
    if (p == 0.0) return nullptr;
    if (!rng.defined()) refuse("rng: needed where p > 0");
    array(rng, "rng", at::kLong, {2}, device);
    return static_cast<const int64_t*>(rng.data_ptr());
}

// The rate as the C functions take it.  One that is too small for fp32 drops nothing, but is not 0: outputs go by that.
float rate(double p) { return p > 0.0 ? std::max((float)p, std::numeric_limits<float>::min()) : 0.0f; }

// The outputs of a call that stores bf16 / fp32 (y) or fp8 in one or both layouts.
struct Result {
    at::Tensor y, q, scales, qt, scales_t;
    int64_t ld = 0, ld_qt = 0;
    void* first() const { return y.defined() ? ptr(y) : ptr(q); }
};
Result result(PyObject* const* v, int64_t type, bool rowwise, bool transpose, int64_t rows, int64_t cols, const at::Device& device,
              const char* plain)
{
    Result r;
    r.y = optional(v[0], plain);
    r.q = optional(v[1], "q");
    r.scales = optional(v[2], "scales");
    r.qt = optional(v[3], "qt");
    r.scales_t = optional(v[4], "scales_t");
    const int64_t shape[2] = {rows, cols};
    if (type == TE_DTYPE_BF16 || type == TE_DTYPE_F32) {
        if (transpose || r.q.defined() || r.scales.defined() || r.qt.defined() || r.scales_t.defined())
            refuse("transpose, q, scales, qt and scales_t belong to fp8 outputs");
        r.ld = make_or_check_rows(r.y, plain, type == TE_DTYPE_BF16 ? kBf16 : kF32, shape, device);
        return r;
    }
    if (!is_fp8(type)) refuse("out_dtype: no type %lld", (long long)type);
    if (r.y.defined()) refuse("%s: fp8 outputs are q and scales", plain);
    if (!rowwise && (r.q.defined() || r.scales.defined())) refuse("q and scales: given with rowwise=False");
    if (!transpose && (r.qt.defined() || r.scales_t.defined())) refuse("qt and scales_t: given with transpose=False");
    if (rowwise) {
        if (cols % 128) refuse("columns must be a multiple of 128 for the fp8 cast (got %lld)", (long long)cols);
        r.ld = make_or_check_rows(r.q, "q", kU8, shape, device);
        make_or_check(r.scales, "scales", kF32, {cols / 128, (rows + 3) / 4 * 4}, device);
    }
    if (transpose) {
        if (rows % 128 || cols % 8)
            refuse("rows must be a multiple of 128 and columns of 8 for the cast of the transpose (got %lld, %lld)", (long long)rows,
                   (long long)cols);
        r.ld_qt = make_or_check_rows(r.qt, "qt", kU8, {cols, rows}, device);
        make_or_check(r.scales_t, "scales_t", kF32, {rows / 128, (cols + 3) / 4 * 4}, device);
    }
    return r;
}

// (x, x_scales, x_dtype, w, w_scales, w_dtype, activation, out_dtype, flags, rowwise, transpose, y, q, scales, qt, scales_t, z, need_z,
//  accum, workspace)
PyObject* gated_fwd(PyObject*, PyObject* const* v, Py_ssize_t n)
{
    return guarded([&] {
        arguments(n, 20);
        const at::Tensor x = required(v[0], "x"), sx = required(v[1], "x_scales"), w = required(v[3], "w"), sw = required(v[4], "w_scales");
        const int64_t xt = integer(v[2]), wt = integer(v[5]), act = integer(v[6]), out = integer(v[7]), flags = integer(v[8]);
        const bool rowwise = truth(v[9]), transpose = truth(v[10]), need_z = truth(v[17]);
        at::Tensor z = optional(v[16], "z"), workspace = optional(v[19], "workspace");
        const int64_t accum = integer(v[18]);
        const at::Device device = x.device();
        operand(x, sx, "x", device);
        operand(w, sw, "w", device);
        const c10::DeviceGuard guard(device);
        const int64_t M = x.size(0), K = x.size(1), H = w.size(0) / 2;
        if (w.size(1) != K || w.size(0) != 2 * H)
            refuse("w: expected shape (2 H, %lld) (got %s)", (long long)K, sizes_of(w.sizes()).c_str());
        if (M < 1 || H < 1 || H % 128) refuse("H must be a multiple of 128, and there must be rows (got %lld, %lld)", (long long)H, (long long)M);
        const Result r = result(v + 11, out, rowwise, transpose, M, H, device, "y");
        int64_t ld_z = 0;
        if (need_z || z.defined()) ld_z = make_or_check_rows(z, "z", kBf16, {M, 2 * H}, device);
        workspace_for(workspace, transpose && M > 128 ? 0 : lib.gated_fwd_workspace_bytes(M, H, K, (te_dtype_t)out), device);
        check(lib.gated_fwd(ptr(x), ptr<float>(sx), (te_dtype_t)xt, ptr(w), ptr<float>(sw), (te_dtype_t)wt, M, H, K, (te_activation_t)act,
                            r.first(), (te_dtype_t)out, r.ld, (uint32_t)flags, ptr<float>(r.scales), ptr(r.qt), r.ld_qt,
                            ptr<float>(r.scales_t), ptr(z), ld_z, ptr(workspace), bytes(workspace), (te_accum_t)accum, stream_of(device)));
        return tuple_of({r.y, r.q, r.scales, r.qt, r.scales_t, z});
    });
}

// (dy, dy_scales, dy_dtype, wt, wt_scales, wt_dtype, z, activation, out_dtype, flags, rowwise, transpose, dz, q, scales, qt, scales_t, accum)
PyObject* gated_dgrad(PyObject*, PyObject* const* v, Py_ssize_t n)
{
    return guarded([&] {
        arguments(n, 18);
        const at::Tensor dy = required(v[0], "dy"), sdy = required(v[1], "dy_scales"), wt = required(v[3], "wt"),
                         swt = required(v[4], "wt_scales"), z = required(v[6], "z");
        const int64_t dt = integer(v[2]), wtt = integer(v[5]), act = integer(v[7]), out = integer(v[8]), flags = integer(v[9]);
        const bool rowwise = truth(v[10]), transpose = truth(v[11]);
        const int64_t accum = integer(v[17]);
        const at::Device device = dy.device();
        operand(dy, sdy, "dy", device);
        operand(wt, swt, "wt", device);
        const c10::DeviceGuard guard(device);
        const int64_t M = dy.size(0), K = dy.size(1), H = wt.size(0);
        if (wt.size(1) != K) refuse("wt: expected shape (H, %lld) (got %s)", (long long)K, sizes_of(wt.sizes()).c_str());
        if (M < 1 || H < 1 || H % 128) refuse("H must be a multiple of 128, and there must be rows (got %lld, %lld)", (long long)H, (long long)M);
        const int64_t ld_z = typed_rows(z, "z", kBf16, {M, 2 * H}, device);
        const Result r = result(v + 12, out, rowwise, transpose, M, 2 * H, device, "dz");
        check(lib.gated_dgrad(ptr(dy), ptr<float>(sdy), (te_dtype_t)dt, ptr(wt), ptr<float>(swt), (te_dtype_t)wtt, M, H, K,
                              (te_activation_t)act, ptr(z), ld_z, r.first(), (te_dtype_t)out, r.ld, (uint32_t)flags, ptr<float>(r.scales),
                              ptr(r.qt), r.ld_qt, ptr<float>(r.scales_t), (te_accum_t)accum, stream_of(device)));
        return tuple_of({r.y, r.q, r.scales, r.qt, r.scales_t});
    });
}

// (x, gamma, beta, eps, residual, p, rng, out_dtype, flags, rowwise, transpose, h, mean, rstd, y, q, scales, qt, scales_t)
PyObject* layernorm_fwd(PyObject*, PyObject* const* v, Py_ssize_t n)
{
    return guarded([&] {
        arguments(n, 19);
        const at::Tensor x = required(v[0], "x"), gamma = required(v[1], "gamma"), beta = optional(v[2], "beta"),
                         residual = optional(v[4], "residual"), rng = optional(v[6], "rng");
        const double eps = number(v[3]), p = number(v[5]);
        const int64_t out = integer(v[7]), flags = integer(v[8]);
        const bool rowwise = truth(v[9]), transpose = truth(v[10]);
        at::Tensor h = optional(v[11], "h"), mean = optional(v[12], "mean"), rstd = optional(v[13], "rstd");
        const int64_t ld_x = matrix(x, "x");
        const int64_t rows = x.size(0), cols = x.size(1);
        const at::Device device = x.device();
        const c10::DeviceGuard guard(device);
        array(gamma, "gamma", kBf16, {cols}, device);
        if (beta.defined()) array(beta, "beta", kBf16, {cols}, device);
        const int64_t* from = state(rng, p, device);
        int64_t ld_res = 0, ld_h = 0;
        if (residual.defined()) {
            ld_res = float_rows(residual, "residual", {rows, cols}, device);
            ld_h = make_or_check_rows(h, "h", residual.scalar_type(), {rows, cols}, device);
        } else if (h.defined()) {
            refuse("h: given without a residual");
        }
        make_or_check(mean, "mean", kF32, {rows}, device);
        make_or_check(rstd, "rstd", kF32, {rows}, device);
        const Result r = result(v + 14, out, rowwise, transpose, rows, cols, device, "y");
        check(lib.layernorm_fwd(ptr(x), type_of(x), ld_x, ptr(residual), residual.defined() ? type_of(residual) : TE_DTYPE_BF16, ld_res,
                                rate(p), from, ptr(gamma), ptr(beta), (float)eps, rows, cols, ptr(h), ld_h, ptr<float>(mean),
                                ptr<float>(rstd), r.first(), (te_dtype_t)out, r.ld, (uint32_t)flags, ptr<float>(r.scales), ptr(r.qt), r.ld_qt,
                                ptr<float>(r.scales_t), stream_of(device)));
        return tuple_of({h, mean, rstd, r.y, r.q, r.scales, r.qt, r.scales_t});
    });
}

// (dy, h, mean, rstd, gamma, dres, p, rng, dx_dtype, dh, dx, dgamma, dbeta, need_dgamma, need_dbeta, workspace)
PyObject* layernorm_bwd(PyObject*, PyObject* const* v, Py_ssize_t n)
{
    return guarded([&] {
        arguments(n, 16);
        const at::Tensor dy = required(v[0], "dy"), h = required(v[1], "h"), mean = required(v[2], "mean"), rstd = required(v[3], "rstd"),
                         gamma = required(v[4], "gamma"), dres = optional(v[5], "dres"), rng = optional(v[7], "rng");
        const double p = number(v[6]);
        const int64_t dx_type = integer(v[8]);
        at::Tensor dh = optional(v[9], "dh"), dx = optional(v[10], "dx"), dgamma = optional(v[11], "dgamma"), dbeta = optional(v[12], "dbeta"),
                   workspace = optional(v[15], "workspace");
        const bool need_dgamma = truth(v[13]), need_dbeta = truth(v[14]);
        const int64_t ld_h = matrix(h, "h");
        const int64_t rows = h.size(0), cols = h.size(1);
        const int64_t shape[2] = {rows, cols};
        const at::Device device = h.device();
        const c10::DeviceGuard guard(device);
        const int64_t ld_dy = float_rows(dy, "dy", shape, device);
        array(mean, "mean", kF32, {rows}, device);
        array(rstd, "rstd", kF32, {rows}, device);
        array(gamma, "gamma", kBf16, {cols}, device);
        const int64_t* from = state(rng, p, device);
        const int64_t ld_res = dres.defined() ? typed_rows(dres, "dres", h.scalar_type(), shape, device) : 0;
        const int64_t ld_dh = make_or_check_rows(dh, "dh", h.scalar_type(), shape, device);
        int64_t ld_dx = 0;
        if (from) {
            if (dx_type != TE_DTYPE_BF16 && dx_type != TE_DTYPE_F32) refuse("dx_dtype: expected TE_DTYPE_BF16 or TE_DTYPE_F32");
            ld_dx = make_or_check_rows(dx, "dx", dx_type == TE_DTYPE_BF16 ? kBf16 : kF32, shape, device);
        } else if (dx.defined()) {
            refuse("dx: given without dropout (dh is x's gradient too)");
        }
        if (!need_dgamma && dgamma.defined()) refuse("dgamma: given with need_dgamma=False");
        if (!need_dbeta && dbeta.defined()) refuse("dbeta: given with need_dbeta=False");
        if (need_dgamma) make_or_check(dgamma, "dgamma", kF32, {cols}, device);
        if (need_dbeta) make_or_check(dbeta, "dbeta", kF32, {cols}, device);
        if (need_dgamma || need_dbeta) workspace_for(workspace, lib.layernorm_bwd_workspace_bytes(rows, cols), device);
        check(lib.layernorm_bwd(ptr(dy), type_of(dy), ld_dy, ptr(h), type_of(h), ld_h, ptr<float>(mean), ptr<float>(rstd), ptr(gamma), rows,
                                cols, ptr(dres), ld_res, ptr(dh), ld_dh, rate(p), from, ptr(dx), (te_dtype_t)dx_type, ld_dx,
                                ptr<float>(dgamma), ptr<float>(dbeta), ptr(workspace), bytes(workspace), stream_of(device)));
        return tuple_of({dh, dx, dgamma, dbeta});
    });
}

// (x, p, rng, residual, out_dtype, out): out_dtype 0: the residual's type, or x's
PyObject* dropout(PyObject*, PyObject* const* v, Py_ssize_t n)
{
    return guarded([&] {
        arguments(n, 6);
        const at::Tensor x = required(v[0], "x"), rng = optional(v[2], "rng"), residual = optional(v[3], "residual");
        const double p = number(v[1]);
        int64_t type = integer(v[4]);
        at::Tensor out = optional(v[5], "out");
        const int64_t ld_x = matrix(x, "x");
        const int64_t shape[2] = {x.size(0), x.size(1)};
        const at::Device device = x.device();
        const c10::DeviceGuard guard(device);
        const int64_t* from = state(rng, p, device);
        const int64_t ld_res = residual.defined() ? float_rows(residual, "residual", shape, device) : 0;
        if (type == 0) type = out.defined() && is_float(out) ? type_of(out) : type_of(residual.defined() ? residual : x);
        if (type != TE_DTYPE_BF16 && type != TE_DTYPE_F32) refuse("out_dtype: expected TE_DTYPE_BF16 or TE_DTYPE_F32");
        const int64_t ld_out = make_or_check_rows(out, "out", type == TE_DTYPE_BF16 ? kBf16 : kF32, shape, device);
        check(lib.dropout(ptr(x), type_of(x), ld_x, ptr(residual), residual.defined() ? type_of(residual) : TE_DTYPE_BF16, ld_res, shape[0],
                          shape[1], rate(p), from, ptr(out), (te_dtype_t)type, ld_out, stream_of(device)));
        return wrap(out);
    });
}

PyObject* bind(PyObject*, PyObject* const* v, Py_ssize_t n) { return bind_library(lib, v, n); }

PyMethodDef methods[] = {TE_METHOD(bind),          TE_METHOD(gated_fwd), TE_METHOD(gated_dgrad),        TE_METHOD(layernorm_fwd),
                         TE_METHOD(layernorm_bwd), TE_METHOD(dropout),   {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_te_block", "Marshalling of the calls of a gated block's operators.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__te_block(void) { return PyModule_Create(&module); }
