// The Python side of the operators around the GEMMs (te_ops.h): checks what the C ABI cannot see of a
// tensor (where it lives, its type, shape and strides), allocates the outputs that are not given, and
// calls the C function.  The calls of few tokens are bound by the host, and these checks in Python cost
// more than their kernels take: the norm of one token took 13.1 us a call so and takes 8.3 us here, the
// router of four tokens 7.6 and 5.1 us, clipping 30 small tensors 28.6 and 8.8 us.
//
// The C functions are those of the library that the package has loaded (bind()); this module
// links to PyTorch only.  Refusals raise the package's TeFp8Error.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <string>
#include <vector>

#include "te_ops.h"

namespace {

struct Library {
    decltype(&te_rmsnorm_fwd) rmsnorm_fwd;
    decltype(&te_rmsnorm_bwd) rmsnorm_bwd;
    decltype(&te_rmsnorm_bwd_workspace_bytes) rmsnorm_bwd_workspace_bytes;
    decltype(&te_moe_router_fwd) moe_router_fwd;
    decltype(&te_moe_router_bwd) moe_router_bwd;
    decltype(&te_moe_router_workspace_bytes) moe_router_workspace_bytes;
    decltype(&te_grad_norm_clip) grad_norm_clip;
    decltype(&te_grad_norm_workspace_bytes) grad_norm_workspace_bytes;
    decltype(&te_status_string) status_string;
    decltype(&te_last_error_message) last_error_message;
} lib{};
PyObject* error_class = nullptr;      // TeFp8Error(status, message)
PyObject* memory_error = nullptr;    // torch.OutOfMemoryError
PyObject* current_stream = nullptr;   // device index -> stream handle

struct Refusal {
    int status;
    std::string message;
};
struct PythonError {};   // one is set already

[[noreturn]] void refuse(const char* fmt, ...) __attribute__((format(printf, 1, 2)));
void refuse(const char* fmt, ...)
{
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    throw Refusal{TE_ERR_INVALID_ARGUMENT, buf};
}

void check(te_status_t status)
{
    if (status != TE_OK)
        throw Refusal{status, std::string(lib.status_string(status)) + ": " + lib.last_error_message()};
}

// Runs a call's body; its exceptions become Python's.
template <class F>
PyObject* guarded(F body)
{
    try {
        if (!lib.rmsnorm_fwd) refuse("the library is not bound");
        return body();
    } catch (const PythonError&) {
    } catch (const Refusal& r) {
        if (PyObject* args = Py_BuildValue("(is)", r.status, r.message.c_str())) {
            PyErr_SetObject(error_class, args);
            Py_DECREF(args);
        }
    } catch (const c10::OutOfMemoryError& e) {
        PyErr_SetString(memory_error, e.what_without_backtrace());   // (as torch.empty)
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    return nullptr;
}

constexpr auto kBf16 = at::kBFloat16;
constexpr auto kF32 = at::kFloat;
constexpr auto kU8 = at::kByte;
constexpr auto kI32 = at::kInt;

bool is_float(const at::Tensor& t) { return t.scalar_type() == kBf16 || t.scalar_type() == kF32; }
te_dtype_t type_of(const at::Tensor& t) { return t.scalar_type() == kBf16 ? TE_DTYPE_BF16 : TE_DTYPE_F32; }

std::string sizes_of(at::IntArrayRef s)
{
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + ")";
}

// A tensor argument; an undefined one for None.
at::Tensor optional(PyObject* o, const char* name)
{
    if (o == Py_None) return at::Tensor();
    if (!THPVariable_Check(o)) refuse("%s: expected a tensor", name);
    return THPVariable_Unpack(o);
}
at::Tensor required(PyObject* o, const char* name)
{
    if (!THPVariable_Check(o)) refuse("%s: expected a tensor", name);
    return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError();
    return v;
}
double number(PyObject* o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PythonError();
    return v;
}
bool truth(PyObject* o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw PythonError();
    return v != 0;
}

// The row stride of a matrix whose rows are consecutive elements and do not overlap.  (That of a
// single row is of no meaning; fp8 rows want a multiple of 16.)
int64_t row_stride(const at::Tensor& t, const char* name)
{
    const int64_t rows = t.size(0), cols = t.size(1);
    if (t.numel() && ((cols > 1 && t.stride(1) != 1) || (rows > 1 && t.stride(0) < cols)))
        refuse("%s: expected rows of consecutive elements that do not overlap (strides %s)", name, sizes_of(t.strides()).c_str());
    return rows > 1 ? t.stride(0) : (cols + 15) / 16 * 16;
}

// What is no bf16 or fp32 matrix on the GPU is refused; returns the row stride.
int64_t matrix(const at::Tensor& t, const char* name)
{
    if (!t.is_cuda() || t.dim() != 2) refuse("%s: expected a matrix on the GPU", name);
    if (!is_float(t)) refuse("%s: expected torch.bfloat16 or torch.float32 (got %s)", name, c10::toString(t.scalar_type()));
    return row_stride(t, name);
}

void same(const at::Tensor& t, const char* name, at::IntArrayRef shape, const at::Device& device)
{
    if (t.device() != device) refuse("%s: expected a tensor on %s", name, device.str().c_str());
    if (t.sizes() != shape) refuse("%s: expected shape %s (got %s)", name, sizes_of(shape).c_str(), sizes_of(t.sizes()).c_str());
}
void typed(const at::Tensor& t, const char* name, at::ScalarType type)
{
    if (t.scalar_type() != type) refuse("%s: expected %s (got %s)", name, c10::toString(type), c10::toString(t.scalar_type()));
}

// A contiguous tensor of the type and shape on the device.
void array(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, const at::Device& device)
{
    same(t, name, shape, device);
    typed(t, name, type);
    if (!t.is_contiguous()) refuse("%s: expected a contiguous tensor", name);
}
// A matrix of the shape on the device, of bf16 or fp32 or of one type, at any row stride; returns that.
int64_t float_rows(const at::Tensor& t, const char* name, at::IntArrayRef shape, const at::Device& device)
{
    same(t, name, shape, device);
    if (!is_float(t)) refuse("%s: expected torch.bfloat16 or torch.float32 (got %s)", name, c10::toString(t.scalar_type()));
    return row_stride(t, name);
}
int64_t typed_rows(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, const at::Device& device)
{
    same(t, name, shape, device);
    typed(t, name, type);
    return row_stride(t, name);
}

// (PyTorch's own allocation function for the GPU, without the dispatcher in front of it: with four to seven
// outputs a call the dispatcher is a tenth of a small call's time: one token's norm takes 9.2 us with it and 8.4
// without, the router with its loss 11.8 and 10.5.)
at::Tensor make(at::IntArrayRef shape, at::ScalarType type, const at::Device& device)
{
    return at::detail::empty_cuda(shape, type, device, std::nullopt);
}
void make_or_check(at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, const at::Device& device)
{
    if (t.defined()) array(t, name, type, shape, device);
    else t = make(shape, type, device);
}
int64_t make_or_check_rows(at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, const at::Device& device)
{
    if (t.defined()) return typed_rows(t, name, type, shape, device);
    t = make(shape, type, device);
    return shape[1];
}
void workspace_for(at::Tensor& t, int64_t need, const at::Device& device)
{
    if (t.defined()) {
        if (t.device() != device || !t.is_contiguous()) refuse("workspace: expected a contiguous tensor on %s", device.str().c_str());
    } else if (need > 0) {
        t = make({need}, kU8, device);
    }
}

template <class T = void>
T* ptr(const at::Tensor& t)
{
    return t.defined() ? static_cast<T*>(t.data_ptr()) : nullptr;
}
int64_t bytes(const at::Tensor& t) { return t.defined() ? (int64_t)t.nbytes() : 0; }

// The device's current stream: outputs and workspaces are allocated for it, so work on another one would
// race with its earlier users of that memory.
hipStream_t stream_of(const at::Device& device)
{
    PyObject* index = PyLong_FromLong(device.index());
    if (!index) throw PythonError();
    PyObject* handle = PyObject_CallOneArg(current_stream, index);
    Py_DECREF(index);
    if (!handle) throw PythonError();
    void* p = PyLong_AsVoidPtr(handle);
    Py_DECREF(handle);
    if (!p && PyErr_Occurred()) throw PythonError();
    return static_cast<hipStream_t>(p);
}

PyObject* wrap(const at::Tensor& t)
{
    if (!t.defined()) Py_RETURN_NONE;
    PyObject* o = THPVariable_Wrap(t);
    if (!o) throw PythonError();
    return o;
}
PyObject* tuple_of(std::initializer_list<at::Tensor> ts)
{
    PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
    if (!r) throw PythonError();
    Py_ssize_t i = 0;
    try {
        for (const at::Tensor& t : ts) PyTuple_SET_ITEM(r, i++, wrap(t));
    } catch (...) {
        Py_DECREF(r);
        throw;
    }
    return r;
}

void arguments(Py_ssize_t have, Py_ssize_t want)
{
    if (have != want) refuse("expected %zd arguments (got %zd)", want, have);
}

// (x, gamma, eps, residual, out_dtype, flags, rowwise, transpose, h, rstd, y, q, scales, qt, scales_t)
PyObject* rmsnorm_fwd(PyObject*, PyObject* const* v, Py_ssize_t n)
{
    return guarded([&] {
        arguments(n, 15);
        const at::Tensor x = required(v[0], "x"), gamma = required(v[1], "gamma"), residual = optional(v[3], "residual");
        const double eps = number(v[2]);
        const int64_t out = integer(v[4]), flags = integer(v[5]);
        const bool rowwise = truth(v[6]), transpose = truth(v[7]);
        at::Tensor h = optional(v[8], "h"), rstd = optional(v[9], "rstd"), y = optional(v[10], "y"), q = optional(v[11], "q"),
                   scales = optional(v[12], "scales"), qt = optional(v[13], "qt"), scales_t = optional(v[14], "scales_t");
        const int64_t ld_x = matrix(x, "x");
        const int64_t rows = x.size(0), cols = x.size(1);
        const int64_t shape[2] = {rows, cols};
        const at::Device device = x.device();
        const c10::DeviceGuard guard(device);
        array(gamma, "gamma", kBf16, {cols}, device);
        int64_t ld_res = 0, ld_h = 0, ld_y = 0, ld_qt = 0;
        if (residual.defined()) {
            ld_res = float_rows(residual, "residual", shape, device);
            ld_h = make_or_check_rows(h, "h", residual.scalar_type(), shape, device);
        } else if (h.defined()) {
            refuse("h: given without a residual");
        }
        make_or_check(rstd, "rstd", kF32, {rows}, device);
        if (out == TE_DTYPE_BF16 || out == TE_DTYPE_F32) {
            if (transpose || q.defined() || scales.defined() || qt.defined() || scales_t.defined())
                refuse("transpose, q, scales, qt and scales_t belong to fp8 outputs");
            ld_y = make_or_check_rows(y, "y", out == TE_DTYPE_BF16 ? kBf16 : kF32, shape, device);
        } else {
            if (out != TE_DTYPE_E4M3 && out != TE_DTYPE_E5M2) refuse("out_dtype: no type %lld", (long long)out);
            if (y.defined()) refuse("y: fp8 outputs are q and scales");
            if (!rowwise && (q.defined() || scales.defined())) refuse("q and scales: given with rowwise=False");
            if (!transpose && (qt.defined() || scales_t.defined())) refuse("qt and scales_t: given with transpose=False");
            if (rowwise) {
                if (cols % 128) refuse("cols must be a multiple of 128 for the fp8 cast (got %lld)", (long long)cols);
                ld_y = make_or_check_rows(q, "q", kU8, shape, device);
                make_or_check(scales, "scales", kF32, {cols / 128, (rows + 3) / 4 * 4}, device);
            }
            if (transpose) {
                if (rows % 128 || cols % 8)
                    refuse("rows must be a multiple of 128 and cols of 8 for the cast of the transpose (got %lld, %lld)",
                           (long long)rows, (long long)cols);
                ld_qt = make_or_check_rows(qt, "qt", kU8, {cols, rows}, device);
                make_or_check(scales_t, "scales_t", kF32, {rows / 128, (cols + 3) / 4 * 4}, device);
            }
        }
        check(lib.rmsnorm_fwd(ptr(x), type_of(x), ld_x, ptr(residual), residual.defined() ? type_of(residual) : TE_DTYPE_BF16, ld_res,
                              ptr(gamma), (float)eps, rows, cols, ptr(h), ld_h, ptr<float>(rstd), y.defined() ? ptr(y) : ptr(q),
                              (te_dtype_t)out, ld_y, (uint32_t)flags, ptr<float>(scales), ptr(qt), ld_qt, ptr<float>(scales_t),
                              stream_of(device)));
        return tuple_of({h, rstd, y, q, scales, qt, scales_t});
    });
}

// (dy, h, rstd, gamma, dres, dh, dgamma, need_dgamma, workspace)
PyObject* rmsnorm_bwd(PyObject*, PyObject* const* v, Py_ssize_t n)
{
    return guarded([&] {
        arguments(n, 9);
        const at::Tensor dy = required(v[0], "dy"), h = required(v[1], "h"), rstd = required(v[2], "rstd"),
                         gamma = required(v[3], "gamma"), dres = optional(v[4], "dres");
        at::Tensor dh = optional(v[5], "dh"), dgamma = optional(v[6], "dgamma"), workspace = optional(v[8], "workspace");
        const bool need_dgamma = truth(v[7]);
        const int64_t ld_h = matrix(h, "h");
        const int64_t rows = h.size(0), cols = h.size(1);
        const int64_t shape[2] = {rows, cols};
        const at::Device device = h.device();
        const c10::DeviceGuard guard(device);
        const int64_t ld_dy = float_rows(dy, "dy", shape, device);
        array(rstd, "rstd", kF32, {rows}, device);
        array(gamma, "gamma", kBf16, {cols}, device);
        const int64_t ld_res = dres.defined() ? typed_rows(dres, "dres", h.scalar_type(), shape, device) : 0;
        const int64_t ld_dh = make_or_check_rows(dh, "dh", h.scalar_type(), shape, device);
        if (need_dgamma) {
            make_or_check(dgamma, "dgamma", kF32, {cols}, device);
            workspace_for(workspace, lib.rmsnorm_bwd_workspace_bytes(rows, cols), device);
        } else if (dgamma.defined()) {
            refuse("dgamma: given with need_dgamma=False");
        }
        check(lib.rmsnorm_bwd(ptr(dy), type_of(dy), ld_dy, ptr(h), type_of(h), ld_h, ptr<float>(rstd), ptr(gamma), rows, cols,
                              ptr(dres), ld_res, ptr(dh), ld_dh, ptr<float>(dgamma), ptr(workspace), bytes(workspace),
                              stream_of(device)));
        return tuple_of({dh, dgamma});
    });
}

// (logits, top_k, renormalize, token_mask, loss, need_lse, workspace)
PyObject* moe_router_fwd(PyObject*, PyObject* const* v, Py_ssize_t n)
{
    return guarded([&] {
        arguments(n, 7);
        const at::Tensor logits = required(v[0], "logits"), mask = optional(v[3], "token_mask");
        const int64_t top_k = integer(v[1]);
        const bool renormalize = truth(v[2]), loss = truth(v[4]), need_lse = truth(v[5]);
        at::Tensor workspace = optional(v[6], "workspace"), lse, counts, routed, value;
        const int64_t ld = matrix(logits, "logits");
        const int64_t tokens = logits.size(0), experts = logits.size(1);
        const at::Device device = logits.device();
        const c10::DeviceGuard guard(device);
        if (top_k < 1 || top_k > experts)
            refuse("top_k must be in [1, experts] (got %lld of %lld)", (long long)top_k, (long long)experts);
        if (mask.defined()) array(mask, "token_mask", mask.scalar_type() == kU8 ? kU8 : at::kBool, {tokens}, device);
        const at::Tensor index = make({tokens, top_k}, kI32, device), weight = make({tokens, top_k}, kF32, device);
        if (need_lse) lse = make({tokens}, kF32, device);
        if (loss) {
            counts = make({experts}, kI32, device);
            routed = make({1}, kI32, device);
            value = make({1}, kF32, device);
            workspace_for(workspace, lib.moe_router_workspace_bytes(tokens, experts), device);
        }
        check(lib.moe_router_fwd(ptr(logits), type_of(logits), ld, tokens, experts, (int32_t)top_k, renormalize, ptr<uint8_t>(mask),
                                 ptr<int32_t>(index), ptr<float>(weight), ptr<float>(lse), ptr<int32_t>(counts),
                                 ptr<int32_t>(routed), ptr<float>(value), ptr(workspace), bytes(workspace),
                                 stream_of(device)));
        return tuple_of({index, weight, lse, counts, routed, value});
    });
}

// (logits, index, lse, counts, routed, d_weight, d_loss, renormalize, d_logits)
PyObject* moe_router_bwd(PyObject*, PyObject* const* v, Py_ssize_t n)
{
    return guarded([&] {
        arguments(n, 9);
        const at::Tensor logits = required(v[0], "logits"), index = required(v[1], "index"), lse = required(v[2], "lse"),
                         d_weight = optional(v[5], "d_weight"), d_loss = optional(v[6], "d_loss");
        const bool renormalize = truth(v[7]);
        at::Tensor d_logits = optional(v[8], "d_logits"), counts, routed;
        const int64_t ld = matrix(logits, "logits");
        const int64_t tokens = logits.size(0), experts = logits.size(1);
        const at::Device device = logits.device();
        const c10::DeviceGuard guard(device);
        if (index.dim() != 2) refuse("index: expected a matrix");
        const int64_t top_k = index.size(1);
        array(index, "index", kI32, {tokens, top_k}, device);
        array(lse, "lse", kF32, {tokens}, device);
        if (d_weight.defined()) array(d_weight, "d_weight", kF32, {tokens, top_k}, device);
        if (d_loss.defined()) {
            if (d_loss.numel() != 1) refuse("d_loss: expected one number");
            array(d_loss, "d_loss", kF32, d_loss.sizes(), device);
            counts = required(v[3], "counts");
            routed = required(v[4], "routed");
            array(counts, "counts", kI32, {experts}, device);
            array(routed, "routed", kI32, {1}, device);
        }
        const int64_t shape[2] = {tokens, experts};
        const int64_t ld_d = make_or_check_rows(d_logits, "d_logits", logits.scalar_type(), shape, device);
        check(lib.moe_router_bwd(ptr(logits), type_of(logits), ld, tokens, experts, (int32_t)std::min<int64_t>(top_k, INT32_MAX),
                                 renormalize, ptr<int32_t>(index), ptr<float>(lse), ptr<float>(d_weight), ptr<int32_t>(counts),
                                 ptr<int32_t>(routed), ptr<float>(d_loss), ptr(d_logits), ld_d, stream_of(device)));
        return wrap(d_logits);
    });
}

// Two tensors whose elements fill one block of memory each, in the same order (contiguous, or permuted alike).
bool same_dense(const at::Tensor& g, const at::Tensor& o)
{
    if (g.is_contiguous() && o.is_contiguous()) return true;
    return g.is_non_overlapping_and_dense() && o.is_non_overlapping_and_dense() && g.strides() == o.strides();
}

// (grads, max_norm, out, norm, workspace): grads and out are lists or tuples, out may be None
PyObject* grad_norm_clip(PyObject*, PyObject* const* v, Py_ssize_t n)
{
    return guarded([&] {
        arguments(n, 5);
        const double max_norm = number(v[1]);
        const bool in_place = v[2] == Py_None;
        if (!(PyList_Check(v[0]) || PyTuple_Check(v[0])) || !(in_place || PyList_Check(v[2]) || PyTuple_Check(v[2])))
            refuse("expected lists of tensors");
        const Py_ssize_t count = PySequence_Fast_GET_SIZE(v[0]);
        if (!in_place && PySequence_Fast_GET_SIZE(v[2]) != count)
            refuse("out: %zd tensors for %zd gradients", PySequence_Fast_GET_SIZE(v[2]), count);
        at::Tensor norm = optional(v[3], "norm"), workspace = optional(v[4], "workspace");
        if (!count && !norm.defined()) refuse("norm: needed where there is no gradient");
        const at::Device device = count ? required(PySequence_Fast_GET_ITEM(v[0], 0), "gradient").device() : norm.device();
        std::vector<te_grad_tensor_t> list((size_t)count);
        for (Py_ssize_t i = 0; i < count; ++i) {
            PyObject *go = PySequence_Fast_GET_ITEM(v[0], i), *oo = in_place ? go : PySequence_Fast_GET_ITEM(v[2], i);
            if (!THPVariable_Check(go) || !THPVariable_Check(oo)) refuse("gradient %zd: expected tensors", i);
            const at::Tensor &g = THPVariable_Unpack(go), &o = THPVariable_Unpack(oo);
            if (!g.is_cuda() || g.device() != device || o.device() != device)
                refuse("gradient %zd: expected gradients and outputs on one GPU", i);
            if (!is_float(g) || !is_float(o)) refuse("gradient %zd: expected torch.bfloat16 or torch.float32", i);
            if (g.sizes() != o.sizes()) refuse("gradient %zd: output of another shape", i);
            if (!same_dense(g, o)) refuse("gradient %zd: expected dense tensors of one layout", i);
            list[(size_t)i] = te_grad_tensor_t{g.data_ptr(), o.data_ptr(), g.numel(), type_of(g), type_of(o)};
        }
        if (!device.is_cuda()) refuse("norm: expected a tensor on the GPU");
        const c10::DeviceGuard guard(device);
        make_or_check(norm, "norm", kF32, {1}, device);
        workspace_for(workspace, lib.grad_norm_workspace_bytes(count), device);
        check(lib.grad_norm_clip(list.data(), count, (float)max_norm, ptr<float>(norm), ptr(workspace), bytes(workspace),
                                 stream_of(device)));
        return wrap(norm);
    });
}

// (error class, torch's out-of-memory class, current stream's function, addresses of the C functions in Library's order)
PyObject* bind(PyObject*, PyObject* const* v, Py_ssize_t n)
{
    constexpr Py_ssize_t kFunctions = sizeof(Library) / sizeof(void*);
    if (n != 3 + kFunctions) {
        PyErr_SetString(PyExc_TypeError, "bind: wrong number of arguments");
        return nullptr;
    }
    void* at[kFunctions];
    for (Py_ssize_t i = 0; i < kFunctions; ++i) {
        at[i] = PyLong_AsVoidPtr(v[3 + i]);
        if (!at[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: null function");
            return nullptr;
        }
    }
    memcpy(&lib, at, sizeof lib);
    Py_INCREF(v[0]);
    Py_XSETREF(error_class, v[0]);
    Py_INCREF(v[1]);
    Py_XSETREF(memory_error, v[1]);
    Py_INCREF(v[2]);
    Py_XSETREF(current_stream, v[2]);
    Py_RETURN_NONE;
}

#define TE_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {TE_METHOD(bind),           TE_METHOD(rmsnorm_fwd),    TE_METHOD(rmsnorm_bwd), TE_METHOD(moe_router_fwd),
                         TE_METHOD(moe_router_bwd), TE_METHOD(grad_norm_clip), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_te_ops", "Marshalling of the operators' calls.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__te_ops(void) { return PyModule_Create(&module); }
