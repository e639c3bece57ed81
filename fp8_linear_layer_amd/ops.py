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
import struct
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


# (PyTorch's handle of the stream without the Stream object around it, whose making costs as much as a launch)
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else \
    lambda index: torch.cuda.current_stream(index).cuda_stream


def _stream(stream, device):
    return _raw_stream(device.index) if stream is None else stream.cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _tensor(t, name, dtype, shape, device):
    """Refuse a tensor that is not a contiguous one of the type and shape on the device."""
    if not isinstance(t, torch.Tensor) or t.device != device:
        _refuse(f"{name}: expected a tensor on {device}")
    if t.dtype is not dtype:
        _refuse(f"{name}: expected {dtype} (got {t.dtype})")
    if t.shape != shape:
        _refuse(f"{name}: expected shape {shape} (got {tuple(t.shape)})")
    if not t.is_contiguous():
        _refuse(f"{name}: expected a contiguous tensor")


def _rows(t, name, dtypes, shape, device):
    """The same for a matrix whose rows may lie at any stride; returns the stride."""
    if not isinstance(t, torch.Tensor) or t.device != device:
        _refuse(f"{name}: expected a tensor on {device}")
    if t.dtype not in dtypes:
        _refuse(f"{name}: expected {' or '.join(map(str, dtypes))} (got {t.dtype})")
    if t.shape != shape:
        _refuse(f"{name}: expected shape {shape} (got {tuple(t.shape)})")
    return _ld(t, name)


def _matrix(t, name):
    """Refuse what is no bf16 or fp32 matrix on the GPU with rows of consecutive elements."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 2:
        _refuse(f"{name}: expected a matrix on the GPU")
    if t.dtype not in _TYPE:
        _refuse(f"{name}: expected torch.bfloat16 or torch.float32 (got {t.dtype})")
    return _ld(t, name)


def _ld(t, name):
    """The row stride.  (That of a single row is of no meaning; fp8 rows want a multiple of 16.)"""
    rows, cols = t.shape
    ld, one = t.stride()
    if t.numel() and ((cols > 1 and one != 1) or (rows > 1 and ld < cols)):
        _refuse(f"{name}: expected rows of consecutive elements that do not overlap (strides {t.stride()})")
    return ld if rows > 1 else (cols + 15) // 16 * 16


def _new(shape, dtype, device):
    return torch.empty_strided(shape, (shape[1], 1) if len(shape) == 2 else (1,), dtype=dtype, device=device)


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
    lib = _bound or _lib()
    ld_x = _matrix(x, "x")
    shape = rows, cols = x.shape
    device = x.device
    _tensor(gamma, "gamma", torch.bfloat16, (cols,), device)
    ld_res = ld_h = ld_y = ld_qt = 0
    if residual is not None:
        ld_res = _rows(residual, "residual", _FLOATS, shape, device)
        if h is None:
            h, ld_h = _new(shape, residual.dtype, device), cols
        else:
            ld_h = _rows(h, "h", (residual.dtype,), shape, device)
    elif h is not None:
        _refuse("h: given without a residual")
    if rstd is None:
        rstd = _new((rows,), torch.float32, device)
    else:
        _tensor(rstd, "rstd", torch.float32, (rows,), device)
    main = None
    if out_dtype == _BF16 or out_dtype == _F32:
        if transpose or q is not None or scales is not None or qt is not None or scales_t is not None:
            _refuse("transpose, q, scales, qt and scales_t belong to fp8 outputs")
        if y is None:
            y, ld_y = _new(shape, _TORCH[out_dtype], device), cols
        else:
            ld_y = _rows(y, "y", (_TORCH[out_dtype],), shape, device)
        main = y
    else:
        if out_dtype not in _TORCH:
            _refuse(f"out_dtype: no type {out_dtype}")
        if y is not None:
            _refuse("y: fp8 outputs are q and scales")
        if rowwise:
            if cols % 128:
                _refuse(f"cols must be a multiple of 128 for the fp8 cast (got {cols})")
            if q is None:
                q, ld_y = _new(shape, torch.uint8, device), cols
            else:
                ld_y = _rows(q, "q", (torch.uint8,), shape, device)
            main = q
            s_shape = (cols // 128, (rows + 3) // 4 * 4)
            if scales is None:
                scales = _new(s_shape, torch.float32, device)
            else:
                _tensor(scales, "scales", torch.float32, s_shape, device)
        elif q is not None or scales is not None:
            _refuse("q and scales: given with rowwise=False")
        if transpose:
            if rows % 128 or cols % 8:
                _refuse(f"rows must be a multiple of 128 and cols of 8 for the cast of the transpose (got {rows}, {cols})")
            if qt is None:
                qt, ld_qt = _new((cols, rows), torch.uint8, device), rows
            else:
                ld_qt = _rows(qt, "qt", (torch.uint8,), (cols, rows), device)
            t_shape = (rows // 128, (cols + 3) // 4 * 4)
            if scales_t is None:
                scales_t = _new(t_shape, torch.float32, device)
            else:
                _tensor(scales_t, "scales_t", torch.float32, t_shape, device)
        elif qt is not None or scales_t is not None:
            _refuse("qt and scales_t: given with transpose=False")
    status = lib.te_rmsnorm_fwd(
        x.data_ptr(), _TYPE[x.dtype], ld_x, _ptr(residual), 0 if residual is None else _TYPE[residual.dtype], ld_res,
        gamma.data_ptr(), eps, rows, cols, _ptr(h), ld_h, rstd.data_ptr(), _ptr(main), out_dtype, ld_y, flags, _ptr(scales),
        _ptr(qt), ld_qt, _ptr(scales_t), _stream(stream, device))
    if status:
        _te._check(status)
    return RmsNormOutput(h, rstd, y, q, scales, qt, scales_t)


def te_rmsnorm_bwd(dy, h, rstd, gamma, dres=None, dh=None, dgamma=None, need_dgamma=True, workspace=None, stream=None):
    """The norm's gradient: (dh, dgamma) for dy [rows, cols] (bf16 or fp32) and what the norm was of,
    h (x without a residual).  dres (h's type) is added to dh; dh=dres adds in place.  dgamma is
    fp32 [cols], None with need_dgamma=False.  The workspace (bytes) is allocated when not given."""
    lib = _bound or _lib()
    ld_h = _matrix(h, "h")
    shape = rows, cols = h.shape
    device = h.device
    ld_dy = _rows(dy, "dy", _FLOATS, shape, device)
    _tensor(rstd, "rstd", torch.float32, (rows,), device)
    _tensor(gamma, "gamma", torch.bfloat16, (cols,), device)
    ld_res = 0 if dres is None else _rows(dres, "dres", (h.dtype,), shape, device)
    if dh is None:
        dh, ld_dh = _new(shape, h.dtype, device), cols
    else:
        ld_dh = _rows(dh, "dh", (h.dtype,), shape, device)
    if not need_dgamma:
        if dgamma is not None:
            _refuse("dgamma: given with need_dgamma=False")
    else:
        if dgamma is None:
            dgamma = _new((cols,), torch.float32, device)
        else:
            _tensor(dgamma, "dgamma", torch.float32, (cols,), device)
        workspace = _workspace(workspace, lib.te_rmsnorm_bwd_workspace_bytes(rows, cols), device)
    status = lib.te_rmsnorm_bwd(
        dy.data_ptr(), _TYPE[dy.dtype], ld_dy, h.data_ptr(), _TYPE[h.dtype], ld_h, rstd.data_ptr(), gamma.data_ptr(), rows,
        cols, _ptr(dres), ld_res, dh.data_ptr(), ld_dh, _ptr(dgamma), _ptr(workspace), _nbytes(workspace),
        _stream(stream, device))
    if status:
        _te._check(status)
    return dh, dgamma


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def _workspace(given, need, device):
    if given is None:
        return _new((need,), torch.uint8, device) if need else None
    if given.device != device or not given.is_contiguous():
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
    lib = _bound or _lib()
    ld = _matrix(logits, "logits")
    tokens, experts = logits.shape
    device = logits.device
    if not 1 <= top_k <= max(experts, 1):
        _refuse(f"top_k must be in [1, experts] (got {top_k} of {experts})")
    if token_mask is not None and token_mask.dtype is not torch.uint8:
        _tensor(token_mask, "token_mask", torch.bool, (tokens,), device)
    elif token_mask is not None:
        _tensor(token_mask, "token_mask", torch.uint8, (tokens,), device)
    index = _new((tokens, top_k), torch.int32, device)
    weight = _new((tokens, top_k), torch.float32, device)
    lse = _new((tokens,), torch.float32, device) if (loss if need_lse is None else need_lse) else None
    counts = routed = out = None
    if loss:
        counts = _new((experts,), torch.int32, device)
        routed = _new((1,), torch.int32, device)
        out = _new((1,), torch.float32, device)
        workspace = _workspace(workspace, lib.te_moe_router_workspace_bytes(tokens, experts), device)
    status = lib.te_moe_router_fwd(
        logits.data_ptr(), _TYPE[logits.dtype], ld, tokens, experts, top_k, bool(renormalize), _ptr(token_mask),
        index.data_ptr(), weight.data_ptr(), _ptr(lse), _ptr(counts), _ptr(routed), _ptr(out), _ptr(workspace),
        _nbytes(workspace), _stream(stream, device))
    if status:
        _te._check(status)
    return RouterOutput(index, weight, lse, counts, routed, out)


def te_moe_router_bwd(logits, index, lse, counts=None, routed=None, d_weight=None, d_loss=None, renormalize=False,
                      d_logits=None, stream=None):
    """d_logits [tokens, experts] for the gradients of the weights (d_weight, fp32 [tokens, top_k]) and
    of the balance loss (d_loss, fp32 [1] on the GPU, with the forward call's counts and routed)."""
    lib = _bound or _lib()
    ld = _matrix(logits, "logits")
    shape = tokens, experts = logits.shape
    device = logits.device
    if not isinstance(index, torch.Tensor) or index.dim() != 2:
        _refuse("index: expected a matrix")
    top_k = index.shape[1]
    _tensor(index, "index", torch.int32, (tokens, top_k), device)
    _tensor(lse, "lse", torch.float32, (tokens,), device)
    if d_weight is not None:
        _tensor(d_weight, "d_weight", torch.float32, (tokens, top_k), device)
    if d_loss is not None:
        if not isinstance(d_loss, torch.Tensor) or d_loss.numel() != 1:
            _refuse("d_loss: expected one number")
        _tensor(d_loss, "d_loss", torch.float32, d_loss.shape, device)
        _tensor(counts, "counts", torch.int32, (experts,), device)
        _tensor(routed, "routed", torch.int32, (1,), device)
    else:
        counts = routed = None
    if d_logits is None:
        d_logits, ld_d = _new(shape, logits.dtype, device), experts
    else:
        ld_d = _rows(d_logits, "d_logits", (logits.dtype,), shape, device)
    status = lib.te_moe_router_bwd(
        logits.data_ptr(), _TYPE[logits.dtype], ld, tokens, experts, top_k, bool(renormalize), index.data_ptr(),
        lse.data_ptr(), _ptr(d_weight), _ptr(counts), _ptr(routed), _ptr(d_loss), d_logits.data_ptr(), ld_d,
        _stream(stream, device))
    if status:
        _te._check(status)
    return d_logits


_data_ptr, _numel = torch.Tensor.data_ptr, torch.Tensor.numel


class _GradTensor(ctypes.Structure):     # te_grad_tensor_t: four 64-bit words
    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("count", ctypes.c_int64),
                ("grad_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32)]


def te_grad_norm_clip(grads, max_norm, out=None, norm=None, workspace=None, stream=None):
    """norm (fp32 [1]) = the norm over all the gradients together, and out[i] = grads[i] *
    min(1, max_norm / (norm + 1e-6)).  Gradients and outputs are lists of dense bf16 or fp32 tensors,
    each with a type of its own; without out the gradients are clipped in place.  Nothing is copied
    to the host."""
    lib = _bound or _lib()
    grads = list(grads)
    outs = grads if out is None else list(out)
    n = len(grads)
    if len(outs) != n:
        _refuse(f"out: {len(outs)} tensors for {n} gradients")
    if n:
        device = grads[0].device
    else:
        device = torch.device("cuda", torch.cuda.current_device()) if norm is None else norm.device
    # (lists of one property at a time: training steps pass hundreds of tensors, and this is a third of
    # the time that a loop over them with all the checks in it takes)
    if not all([t.is_cuda for t in grads]) or len({t.device for t in grads} | {t.device for t in outs}) > 1:
        _refuse("expected gradients and outputs on one GPU")
    types = [_TYPE.get(t.dtype) for t in grads]
    out_types = types if outs is grads else [_TYPE.get(t.dtype) for t in outs]
    if None in types or None in out_types:
        _refuse(f"expected torch.bfloat16 or torch.float32 (got {({t.dtype for t in grads + outs})})")
    if outs is not grads and [t.shape for t in grads] != [t.shape for t in outs]:
        _refuse("out: expected the gradients' shapes")
    if not (all([t.is_contiguous() for t in grads]) and (outs is grads or all([t.is_contiguous() for t in outs]))):
        for i, (g, o) in enumerate(zip(grads, outs)):
            if not (g.is_contiguous() and o.is_contiguous()) and not _same_dense(g, o):
                _refuse(f"gradient {i}: expected dense tensors of one layout")
    fields = [0] * (4 * n)
    fields[0::4] = map(_data_ptr, grads)
    fields[1::4] = map(_data_ptr, outs)
    fields[2::4] = map(_numel, grads)
    fields[3::4] = [g | o << 32 for g, o in zip(types, out_types)]
    if norm is None:
        norm = _new((1,), torch.float32, device)
    else:
        _tensor(norm, "norm", torch.float32, (1,), device)
    workspace = _workspace(workspace, lib.te_grad_norm_workspace_bytes(n), device)
    status = lib.te_grad_norm_clip(struct.pack(f"{4 * n}q", *fields), n, max_norm, norm.data_ptr(), _ptr(workspace),
                                   _nbytes(workspace), _stream(stream, device))
    if status:
        _te._check(status)
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
