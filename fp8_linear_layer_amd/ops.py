"""Python binding of the operators around the GEMMs (``include/te_ops.h``): the root-mean-square
norm with the residual's addition, the top-k router with its balance loss, and the global gradient
norm with clipping.

Argument marshalling only, as in the package's ``__init__``: every step runs in the HIP kernels of
``libte_fp8.so``.  The C side checks values and alignment; what it cannot see (where a tensor lives,
its type, shape and strides) is checked here before its pointer is passed on.  A refused call raises
``TeFp8Error`` and launches nothing.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

import fp8_linear_layer_amd as _te

_BF16, _F32 = _te.TE_DTYPE_BF16, _te.TE_DTYPE_F32
_TYPE = {torch.bfloat16: _BF16, torch.float32: _F32}
_TORCH = {_BF16: torch.bfloat16, _F32: torch.float32, _te.TE_DTYPE_E4M3: torch.uint8, _te.TE_DTYPE_E5M2: torch.uint8}

EXPORTED = ("te_rmsnorm_fwd", "te_rmsnorm_bwd", "te_rmsnorm_bwd_workspace_bytes", "te_moe_router_fwd",
            "te_moe_router_bwd", "te_moe_router_workspace_bytes", "te_grad_norm_clip", "te_grad_norm_workspace_bytes")

_bound = None


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


def _refuse(message: str):
    raise _te.TeFp8Error(1, message)


def _stream(stream, device):
    return (torch.cuda.current_stream(device) if stream is None else stream).cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _tensor(t, name, dtypes, shape, device, contiguous=True):
    """Refuse a tensor that is not on `device`, of one of the dtypes and of the shape (with
    contiguous=False: rows of consecutive elements at any stride)."""
    if not isinstance(t, torch.Tensor) or t.device != device or not t.is_cuda:
        _refuse(f"{name}: expected a tensor on {device}")
    if t.dtype not in dtypes:
        _refuse(f"{name}: expected {' or '.join(str(d) for d in dtypes)} (got {t.dtype})")
    if tuple(t.shape) != tuple(shape):
        _refuse(f"{name}: expected shape {tuple(shape)} (got {tuple(t.shape)})")
    if contiguous:
        if not t.is_contiguous():
            _refuse(f"{name}: expected a contiguous tensor")
    elif t.numel() and ((shape[1] > 1 and t.stride(1) != 1) or (shape[0] > 1 and t.stride(0) < shape[1])):
        _refuse(f"{name}: expected rows of consecutive elements that do not overlap (strides {t.stride()})")


def _ld(t):
    return max(t.stride(0), t.shape[1]) if t.shape[0] > 1 else _row_ld(t)


def _row_ld(t):
    # (the stride of a single row is of no meaning; fp8 rows want a multiple of 16)
    n = t.shape[1]
    return (n + 15) // 16 * 16


def _matrix(t, name):
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or not t.is_cuda:
        _refuse(f"{name}: expected a matrix on the GPU")
    if t.dtype not in _TYPE:
        _refuse(f"{name}: expected torch.bfloat16 or torch.float32 (got {t.dtype})")
    if t.numel() and ((t.shape[1] > 1 and t.stride(1) != 1) or (t.shape[0] > 1 and t.stride(0) < t.shape[1])):
        _refuse(f"{name}: expected rows of consecutive elements that do not overlap (strides {t.stride()})")


_FLOATS = (torch.bfloat16, torch.float32)


class RmsNormOutput(NamedTuple):
    """What te_rmsnorm_fwd returns; None where the call has no such output."""
    h: torch.Tensor | None         # x + residual, [rows, cols]
    rstd: torch.Tensor             # fp32 [rows]
    y: torch.Tensor | None         # [rows, cols], bf16 or fp32 output
    q: torch.Tensor | None         # uint8 [rows, cols], fp8 output
    scales: torch.Tensor | None    # fp32 [cols/128, scale_ld(rows)]
    qt: torch.Tensor | None        # uint8 [cols, rows]
    scales_t: torch.Tensor | None  # fp32 [rows/128, scale_ld(cols)]


def te_rmsnorm_fwd(x, gamma, eps=1e-5, residual=None, out_dtype=_BF16, flags=0, rowwise=True, transpose=False, h=None,
                   rstd=None, y=None, q=None, scales=None, qt=None, scales_t=None, stream=None) -> RmsNormOutput:
    """h = x + residual (in the residual's type), y = h / rms(h) * gamma, stored by out_dtype as bf16 /
    fp32 (y), or in fp8 as its per-token cast (q, scales; rowwise) and / or the cast of its transpose
    (qt, scales_t; transpose).  x and residual are bf16 or fp32 [rows, cols], gamma bf16 [cols].
    Outputs that are not given are allocated; h=residual adds in place."""
    lib = _lib()
    _matrix(x, "x")
    rows, cols = x.shape
    device = x.device
    _tensor(gamma, "gamma", (torch.bfloat16,), (cols,), device)
    if out_dtype not in _TORCH:
        _refuse(f"out_dtype: no type {out_dtype}")
    fp8 = out_dtype not in (_BF16, _F32)
    if residual is not None:
        _tensor(residual, "residual", _FLOATS, (rows, cols), device, contiguous=False)
        if h is None:
            h = torch.empty((rows, cols), dtype=residual.dtype, device=device)
        else:
            _tensor(h, "h", (residual.dtype,), (rows, cols), device, contiguous=False)
    elif h is not None:
        _refuse("h: given without a residual")
    if rstd is None:
        rstd = torch.empty((rows,), dtype=torch.float32, device=device)
    else:
        _tensor(rstd, "rstd", (torch.float32,), (rows,), device)
    if not fp8:
        if transpose or q is not None or scales is not None or qt is not None or scales_t is not None:
            _refuse("transpose, q, scales, qt and scales_t belong to fp8 outputs")
        if y is None:
            y = torch.empty((rows, cols), dtype=_TORCH[out_dtype], device=device)
        else:
            _tensor(y, "y", (_TORCH[out_dtype],), (rows, cols), device, contiguous=False)
        main = y
    else:
        if y is not None:
            _refuse("y: fp8 outputs are q and scales")
        if (not rowwise and (q is not None or scales is not None)) or \
                (not transpose and (qt is not None or scales_t is not None)):
            _refuse("an fp8 output was given that the call does not write")
        if rowwise:
            if cols % 128:
                _refuse(f"cols must be a multiple of 128 for the fp8 cast (got {cols})")
            if q is None:
                q = torch.empty((rows, cols), dtype=torch.uint8, device=device)
            else:
                _tensor(q, "q", (torch.uint8,), (rows, cols), device, contiguous=False)
            if scales is None:
                scales = torch.empty((cols // 128, (rows + 3) // 4 * 4), dtype=torch.float32, device=device)
            else:
                _tensor(scales, "scales", (torch.float32,), (cols // 128, (rows + 3) // 4 * 4), device)
        if transpose:
            if rows % 128 or cols % 8:
                _refuse(f"rows must be a multiple of 128 and cols of 8 for the cast of the transpose (got {rows}, {cols})")
            if qt is None:
                qt = torch.empty((cols, rows), dtype=torch.uint8, device=device)
            else:
                _tensor(qt, "qt", (torch.uint8,), (cols, rows), device, contiguous=False)
            if scales_t is None:
                scales_t = torch.empty((rows // 128, (cols + 3) // 4 * 4), dtype=torch.float32, device=device)
            else:
                _tensor(scales_t, "scales_t", (torch.float32,), (rows // 128, (cols + 3) // 4 * 4), device)
        main = q
    _te._check(lib.te_rmsnorm_fwd(
        x.data_ptr(), _TYPE[x.dtype], _ld(x), _ptr(residual), _TYPE[residual.dtype] if residual is not None else 0,
        _ld(residual) if residual is not None else 0, gamma.data_ptr(), eps, rows, cols, _ptr(h),
        _ld(h) if h is not None else 0, rstd.data_ptr(), _ptr(main), out_dtype, _ld(main) if main is not None else 0,
        flags, _ptr(scales), _ptr(qt), _ld(qt) if qt is not None else 0, _ptr(scales_t), _stream(stream, device)))
    return RmsNormOutput(h, rstd, y, q, scales, qt, scales_t)


def te_rmsnorm_bwd(dy, h, rstd, gamma, dres=None, dh=None, dgamma=None, need_dgamma=True, workspace=None, stream=None):
    """The norm's gradient: (dh, dgamma) for dy [rows, cols] (bf16 or fp32) and what the norm was of,
    h (x without a residual).  dres (h's type) is added to dh; dh=dres adds in place.  dgamma is
    fp32 [cols], None with need_dgamma=False.  The workspace (bytes) is allocated when not given."""
    lib = _lib()
    _matrix(h, "h")
    rows, cols = h.shape
    device = h.device
    _tensor(dy, "dy", _FLOATS, (rows, cols), device, contiguous=False)
    _tensor(rstd, "rstd", (torch.float32,), (rows,), device)
    _tensor(gamma, "gamma", (torch.bfloat16,), (cols,), device)
    if dres is not None:
        _tensor(dres, "dres", (h.dtype,), (rows, cols), device, contiguous=False)
    if dh is None:
        dh = torch.empty((rows, cols), dtype=h.dtype, device=device)
    else:
        _tensor(dh, "dh", (h.dtype,), (rows, cols), device, contiguous=False)
    if not need_dgamma:
        if dgamma is not None:
            _refuse("dgamma: given with need_dgamma=False")
    else:
        if dgamma is None:
            dgamma = torch.empty((cols,), dtype=torch.float32, device=device)
        else:
            _tensor(dgamma, "dgamma", (torch.float32,), (cols,), device)
        workspace = _workspace(workspace, lib.te_rmsnorm_bwd_workspace_bytes(rows, cols), device)
    _te._check(lib.te_rmsnorm_bwd(
        dy.data_ptr(), _TYPE[dy.dtype], _ld(dy), h.data_ptr(), _TYPE[h.dtype], _ld(h), rstd.data_ptr(),
        gamma.data_ptr(), rows, cols, _ptr(dres), _ld(dres) if dres is not None else 0, dh.data_ptr(), _ld(dh),
        _ptr(dgamma), _ptr(workspace), _nbytes(workspace), _stream(stream, device)))
    return dh, dgamma


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def _workspace(given, need, device):
    if given is None:
        return torch.empty((need,), dtype=torch.uint8, device=device) if need else None
    if not given.is_cuda or given.device != device or not given.is_contiguous():
        _refuse(f"workspace: expected a contiguous tensor on {device}")
    return given


class RouterOutput(NamedTuple):
    """What te_moe_router_fwd returns; None where the call has no such output."""
    index: torch.Tensor           # int32 [tokens, top_k], -1 where the token goes nowhere
    weight: torch.Tensor          # fp32 [tokens, top_k]
    lse: torch.Tensor | None      # fp32 [tokens]
    counts: torch.Tensor | None   # int32 [experts]
    routed: torch.Tensor | None   # int32 [1]
    loss: torch.Tensor | None     # fp32 [1]


def te_moe_router_fwd(logits, top_k, renormalize=False, token_mask=None, loss=False, need_lse=None, workspace=None,
                      stream=None) -> RouterOutput:
    """The top_k experts of each token and their softmax weights (renormalize: divided by their sum);
    logits are bf16 or fp32 [tokens, experts], -inf closes an expert, token_mask (bool or uint8
    [tokens]) leaves tokens out.  With loss also the tokens per expert, the number of routed tokens
    and the balance loss.  lse, which the backward pass needs, comes with loss or need_lse."""
    lib = _lib()
    _matrix(logits, "logits")
    tokens, experts = logits.shape
    device = logits.device
    if not 1 <= top_k <= max(experts, 1):
        _refuse(f"top_k must be in [1, experts] (got {top_k} of {experts})")
    if token_mask is not None:
        _tensor(token_mask, "token_mask", (torch.bool, torch.uint8), (tokens,), device)
    index = torch.empty((tokens, top_k), dtype=torch.int32, device=device)
    weight = torch.empty((tokens, top_k), dtype=torch.float32, device=device)
    lse = torch.empty((tokens,), dtype=torch.float32, device=device) if (loss if need_lse is None else need_lse) else None
    counts = routed = out = None
    if loss:
        counts = torch.empty((experts,), dtype=torch.int32, device=device)
        routed = torch.empty((1,), dtype=torch.int32, device=device)
        out = torch.empty((1,), dtype=torch.float32, device=device)
        workspace = _workspace(workspace, lib.te_moe_router_workspace_bytes(tokens, experts), device)
    _te._check(lib.te_moe_router_fwd(
        logits.data_ptr(), _TYPE[logits.dtype], _ld(logits), tokens, experts, top_k, bool(renormalize),
        _ptr(token_mask), index.data_ptr(), weight.data_ptr(), _ptr(lse), _ptr(counts), _ptr(routed), _ptr(out),
        _ptr(workspace), _nbytes(workspace), _stream(stream, device)))
    return RouterOutput(index, weight, lse, counts, routed, out)


def te_moe_router_bwd(logits, index, lse, counts=None, routed=None, d_weight=None, d_loss=None, renormalize=False,
                      d_logits=None, stream=None):
    """d_logits [tokens, experts] for the gradients of the weights (d_weight, fp32 [tokens, top_k]) and
    of the balance loss (d_loss, fp32 [1] on the GPU, with the forward call's counts and routed)."""
    lib = _lib()
    _matrix(logits, "logits")
    tokens, experts = logits.shape
    device = logits.device
    if not isinstance(index, torch.Tensor) or index.dim() != 2:
        _refuse("index: expected a matrix")
    top_k = index.shape[1]
    _tensor(index, "index", (torch.int32,), (tokens, top_k), device)
    _tensor(lse, "lse", (torch.float32,), (tokens,), device)
    if d_weight is not None:
        _tensor(d_weight, "d_weight", (torch.float32,), (tokens, top_k), device)
    if d_loss is not None:
        if not isinstance(d_loss, torch.Tensor) or d_loss.numel() != 1:
            _refuse("d_loss: expected one number")
        _tensor(d_loss, "d_loss", (torch.float32,), d_loss.shape, device)
        _tensor(counts, "counts", (torch.int32,), (experts,), device)
        _tensor(routed, "routed", (torch.int32,), (1,), device)
    if d_logits is None:
        d_logits = torch.empty((tokens, experts), dtype=logits.dtype, device=device)
    else:
        _tensor(d_logits, "d_logits", (logits.dtype,), (tokens, experts), device, contiguous=False)
    _te._check(lib.te_moe_router_bwd(
        logits.data_ptr(), _TYPE[logits.dtype], _ld(logits), tokens, experts, top_k, bool(renormalize),
        index.data_ptr(), lse.data_ptr(), _ptr(d_weight), _ptr(counts) if d_loss is not None else None,
        _ptr(routed) if d_loss is not None else None, _ptr(d_loss), d_logits.data_ptr(), _ld(d_logits),
        _stream(stream, device)))
    return d_logits


class _GradTensor(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("count", ctypes.c_int64),
                ("grad_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32)]


def te_grad_norm_clip(grads, max_norm, out=None, norm=None, workspace=None, stream=None):
    """norm (fp32 [1]) = the norm over all the gradients together, and out[i] = grads[i] *
    min(1, max_norm / (norm + 1e-6)).  Gradients and outputs are lists of dense bf16 or fp32 tensors,
    each with a type of its own; without out the gradients are clipped in place.  Nothing is copied
    to the host."""
    lib = _lib()
    grads = list(grads)
    outs = grads if out is None else list(out)
    if len(outs) != len(grads):
        _refuse(f"out: {len(outs)} tensors for {len(grads)} gradients")
    device = grads[0].device if grads else torch.device("cuda", torch.cuda.current_device()) if norm is None else norm.device
    arr = (_GradTensor * len(grads))()
    for i, (g, o) in enumerate(zip(grads, outs)):
        kind, okind = _TYPE.get(g.dtype), _TYPE.get(o.dtype)
        if not g.is_cuda or g.device != device or o.device != device:
            _refuse(f"gradient {i}: expected gradient and output on {device if device.type == 'cuda' else 'the GPU'}")
        if kind is None or okind is None:
            _refuse(f"gradient {i}: expected torch.bfloat16 or torch.float32 (got {g.dtype}, {o.dtype})")
        if o is not g and o.shape != g.shape:
            _refuse(f"gradient {i}: output of shape {tuple(o.shape)} for {tuple(g.shape)}")
        if not (g.is_contiguous() and (o is g or o.is_contiguous())) and not _same_dense(g, o):
            _refuse(f"gradient {i}: expected dense tensors of one layout")
        arr[i] = (g.data_ptr(), o.data_ptr(), g.numel(), kind, okind)
    if norm is None:
        norm = torch.empty((1,), dtype=torch.float32, device=device)
    else:
        _tensor(norm, "norm", (torch.float32,), (1,), device)
    workspace = _workspace(workspace, lib.te_grad_norm_workspace_bytes(len(grads)), device)
    _te._check(lib.te_grad_norm_clip(arr, len(grads), max_norm, norm.data_ptr(), _ptr(workspace), _nbytes(workspace),
                                     _stream(stream, device)))
    return norm


def _same_dense(g, o):
    """Two tensors whose elements fill one block of memory each, in the same order (a permuted one)."""
    if g.stride() != o.stride():
        return False
    expect = 1
    for stride, size in sorted((st, sz) for st, sz in zip(g.stride(), g.shape) if sz != 1):
        if stride != expect:
            return False
        expect *= size
    return True
