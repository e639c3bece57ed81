"""Python binding of the operators around the GEMMs (``include/te_ops.h``): the root-mean-square
norm with the residual's addition, the top-k router with its balance loss, and the global gradient
norm with clipping.

Signatures and documentation only: the checks of the tensors, the allocation of outputs and the call
of the C function are native (``csrc/binding.cpp``), and every step of the computation runs in the
HIP kernels of ``libte_fp8.so``.  A refused call raises ``TeFp8Error`` and launches nothing, one whose
outputs find no memory ``torch.OutOfMemoryError``; without the built libraries every call raises.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
from typing import NamedTuple

import torch

import fp8_linear_layer_amd as _te

BINDING_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_te_ops.so")
EXPORTED = ("te_rmsnorm_fwd", "te_rmsnorm_bwd", "te_rmsnorm_bwd_workspace_bytes", "te_moe_router_fwd",
            "te_moe_router_bwd", "te_moe_router_workspace_bytes", "te_grad_norm_clip", "te_grad_norm_workspace_bytes")

_bound = None     # the library with the operators' functions declared
_native = None    # the binding module, calling into that library


class _GradTensor(ctypes.Structure):     # te_grad_tensor_t
    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("count", ctypes.c_int64),
                ("grad_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32)]


def _lib():
    global _bound
    if _bound is None:
        lib = _te.load_library()
        P, I64, U32, I32, I, F = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint32, ctypes.c_int32, ctypes.c_int,
                                  ctypes.c_float)
        for name, restype, argtypes in (
                ("te_rmsnorm_fwd", I, [P, I, I64, P, I, I64, P, F, I64, I64, P, I64, P, P, I, I64, U32, P, P, I64, P, P]),
                ("te_rmsnorm_bwd_workspace_bytes", I64, [I64, I64]),
                ("te_rmsnorm_bwd", I, [P, I, I64, P, I, I64, P, P, I64, I64, P, I64, P, I64, P, P, I64, P]),
                ("te_moe_router_workspace_bytes", I64, [I64, I64]),
                ("te_moe_router_fwd", I, [P, I, I64, I64, I64, I32, I32, P, P, P, P, P, P, P, P, I64, P]),
                ("te_moe_router_bwd", I, [P, I, I64, I64, I64, I32, I32, P, P, P, P, P, P, P, I64, P]),
                ("te_grad_norm_workspace_bytes", I64, [I64]),
                ("te_grad_norm_clip", I, [P, I64, F, P, P, I64, P])):
            f = getattr(lib, name)
            f.restype, f.argtypes = restype, argtypes
        _bound = lib
    return _bound


def _current_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


def _load():
    """The binding module, bound to the library's functions (built in-tree like the library)."""
    global _native
    lib = _lib()
    if not os.path.exists(BINDING_PATH):
        raise RuntimeError(f"{BINDING_PATH} is missing: build it with `python -m fp8_linear_layer_amd.build`")
    spec = importlib.util.spec_from_file_location("_te_ops", BINDING_PATH)
    native = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(native)
    # (PyTorch's plain handle of the current stream, where it has one: the Stream object around it costs as
    # much as a launch)
    native.bind(_te.TeFp8Error, torch.OutOfMemoryError, getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream),
                *[ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in
                  ("te_rmsnorm_fwd", "te_rmsnorm_bwd", "te_rmsnorm_bwd_workspace_bytes", "te_moe_router_fwd",
                   "te_moe_router_bwd", "te_moe_router_workspace_bytes", "te_grad_norm_clip",
                   "te_grad_norm_workspace_bytes", "te_status_string", "te_last_error_message")])
    _native = native
    return native


class RmsNormOutput(NamedTuple):
    """What te_rmsnorm_fwd returns; None where the call has no such output."""
    h: torch.Tensor | None         # x + residual, [rows, cols]
    rstd: torch.Tensor             # fp32 [rows]
    y: torch.Tensor | None         # [rows, cols], bf16 or fp32 output
    q: torch.Tensor | None         # uint8 [rows, cols], fp8 output
    scales: torch.Tensor | None    # fp32 [cols/128, scale_ld(rows)]
    qt: torch.Tensor | None        # uint8 [cols, rows]
    scales_t: torch.Tensor | None  # fp32 [rows/128, scale_ld(cols)]


class RouterOutput(NamedTuple):
    """What te_moe_router_fwd returns; None where the call has no such output."""
    index: torch.Tensor           # int32 [tokens, top_k], -1 where the token goes nowhere
    weight: torch.Tensor          # fp32 [tokens, top_k]
    lse: torch.Tensor | None      # fp32 [tokens]
    counts: torch.Tensor | None   # int32 [experts]
    routed: torch.Tensor | None   # int32 [1]
    loss: torch.Tensor | None     # fp32 [1]


def _call(name, stream, *args):
    """The native call on a given stream: made that stream the current one, so that what the call
    allocates belongs to it too."""
    if stream is None:
        return getattr(_native or _load(), name)(*args)
    with torch.cuda.stream(stream):
        return getattr(_native or _load(), name)(*args)


def te_rmsnorm_fwd(x, gamma, eps=1e-5, residual=None, out_dtype=_te.TE_DTYPE_BF16, flags=0, rowwise=True, transpose=False,
                   h=None, rstd=None, y=None, q=None, scales=None, qt=None, scales_t=None, stream=None) -> RmsNormOutput:
    """h = x + residual (in the residual's type), y = h / rms(h) * gamma, stored by out_dtype as bf16 /
    fp32 (y), or in fp8 as its per-token cast (q, scales; rowwise) and / or the cast of its transpose
    (qt, scales_t; transpose).  x and residual are bf16 or fp32 [rows, cols], gamma bf16 [cols].
    Outputs that are not given are allocated; h=residual adds in place."""
    return RmsNormOutput._make(_call("rmsnorm_fwd", stream, x, gamma, eps, residual, out_dtype, flags, rowwise, transpose,
                                     h, rstd, y, q, scales, qt, scales_t))


def te_rmsnorm_bwd(dy, h, rstd, gamma, dres=None, dh=None, dgamma=None, need_dgamma=True, workspace=None, stream=None):
    """The norm's gradient: (dh, dgamma) for dy [rows, cols] (bf16 or fp32) and what the norm was of,
    h (x without a residual).  dres (h's type) is added to dh; dh=dres adds in place.  dgamma is
    fp32 [cols], None with need_dgamma=False.  The workspace (bytes) is allocated when not given."""
    return _call("rmsnorm_bwd", stream, dy, h, rstd, gamma, dres, dh, dgamma, need_dgamma, workspace)


def te_moe_router_fwd(logits, top_k, renormalize=False, token_mask=None, loss=False, need_lse=None, workspace=None,
                      stream=None) -> RouterOutput:
    """The top_k experts of each token and their softmax weights (renormalize: divided by their sum);
    logits are bf16 or fp32 [tokens, experts], -inf closes an expert, token_mask (bool or uint8
    [tokens]) leaves tokens out.  With loss also the tokens per expert, the number of routed tokens
    and the balance loss.  lse, which the backward pass needs, comes with loss or need_lse."""
    return RouterOutput._make(_call("moe_router_fwd", stream, logits, top_k, renormalize, token_mask, loss,
                                    loss if need_lse is None else need_lse, workspace))


def te_moe_router_bwd(logits, index, lse, counts=None, routed=None, d_weight=None, d_loss=None, renormalize=False,
                      d_logits=None, stream=None):
    """d_logits [tokens, experts] for the gradients of the weights (d_weight, fp32 [tokens, top_k]) and
    of the balance loss (d_loss, fp32 [1] on the GPU, with the forward call's counts and routed)."""
    return _call("moe_router_bwd", stream, logits, index, lse, counts, routed, d_weight, d_loss, renormalize, d_logits)


def te_grad_norm_clip(grads, max_norm, out=None, norm=None, workspace=None, stream=None):
    """norm (fp32 [1]) = the norm over all the gradients together, and out[i] = grads[i] *
    min(1, max_norm / (norm + 1e-6)).  Gradients and outputs are lists of dense bf16 or fp32 tensors,
    each with a type of its own; without out the gradients are clipped in place.  Nothing is copied
    to the host."""
    if type(grads) is not list:
        grads = list(grads)
    if out is not None and type(out) is not list:
        out = list(out)
    if not grads and norm is None:
        with torch.cuda.stream(stream):      # (None: the current one)
            norm = torch.empty((1,), dtype=torch.float32, device="cuda")
    return _call("grad_norm_clip", stream, grads, max_norm, out, norm, workspace)
