"""Training modules on the operators around the GEMMs: the root-mean-square norm with the residual's
addition (RmsNorm), the same in front of an FP8 MLP with the norm writing the MLP's fp8 operands
(Fp8NormMlp), the top-k router with its balance loss (TopKRouter), and the clipping of the gradients
that the modules accumulate (clip_grad_norm).

As in ``linear``: every product, norm, softmax and reduction of forward and backward is a library call;
torch supplies device memory, streams, autograd's bookkeeping, and the casts and additions of the
parameters' small gradient vectors.  The residual stream is handed on explicitly: a
module takes (x, residual), adds them, and returns its output and the sum h, which is the next
module's residual; in the backward pass the gradient of h is added by the norm's backward kernel.
"""
from __future__ import annotations

import torch

from . import (TE_ACCUM_FULL_FP32, TE_DTYPE_BF16, TE_EPI_AUX_PREACT, TE_EPI_BGRAD, TE_EPI_BIAS, TE_EPI_DGELU, TE_EPI_GELU,
               te_cast_fp8_per_token_transpose, te_fp8_gemm_dgrad, te_fp8_gemm_dgrad_deterministic, te_fp8_gemm_fwd,
               te_fp8_wgrad_accum, te_fp8_wgrad_accum_bgrad, te_grad_norm_clip, te_moe_router_bwd, te_moe_router_fwd,
               te_rmsnorm_bwd, te_rmsnorm_fwd)
from .linear import BWD_DTYPE, FWD_DTYPE, Fp8Mlp, _check_dims, _first_order, _fwd_policy, _grad_buffer, _unread


def _to_param(grad32, param):
    """An fp32 gradient as autograd wants it, or None after adding it to the parameter's main_grad."""
    main = getattr(param, "main_grad", None)
    if main is None:
        return grad32.to(param.dtype)
    main.add_(grad32)
    return None


class _RmsNormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, gamma, eps: float):
        ctx.set_materialize_grads(False)
        r = te_rmsnorm_fwd(x, gamma, eps, residual=residual)
        h = x if residual is None else r.h
        ctx.save_for_backward(h, r.rstd, gamma)
        ctx.added, ctx.x_dtype = residual is not None, x.dtype
        return (r.y, h) if residual is not None else (r.y, None)

    @staticmethod
    def backward(ctx, dy, dh_next):
        if dy is None:      # only h was used
            return (dh_next.to(ctx.x_dtype) if dh_next is not None else None), dh_next, None, None
        return _RmsNormFn.gradients(ctx, dy, dh_next)

    @staticmethod
    @_first_order
    def gradients(ctx, dy, dh_next):
        h, rstd, gamma = ctx.saved_tensors
        train = ctx.needs_input_grad[2]      # a frozen weight: no sums, and nothing added to its main_grad
        dh, dgamma = te_rmsnorm_bwd(dy.contiguous(), h, rstd, gamma, dres=dh_next.contiguous() if dh_next is not None else None,
                                    need_dgamma=train)
        return dh.to(ctx.x_dtype), (dh if ctx.added else None), (_to_param(dgamma, gamma) if train else None), None


class RmsNorm(torch.nn.Module):
    """forward(x, residual=None) -> (y, h): h = x + residual in the residual's type (x itself without
    one), y = bf16 h / rms(h) * weight.  With main_grad the weight's gradient is accumulated in fp32
    there and weight.grad stays None."""

    def __init__(self, features, eps=1e-5, device="cuda", main_grad=True):
        super().__init__()
        self.eps = eps
        self.weight = torch.nn.Parameter(torch.ones(features, dtype=torch.bfloat16, device=device))
        if main_grad:
            self.weight.main_grad = torch.zeros((features,), dtype=torch.float32, device=device)

    def forward(self, x, residual=None):
        shp = x.shape
        flat = residual.reshape(-1, shp[-1]) if residual is not None else None
        y, h = _RmsNormFn.apply(x.reshape(-1, shp[-1]), flat, self.weight, self.eps)
        return y.reshape(shp), (x if h is None else h.reshape(shp))


class _Fp8NormMlpFn(torch.autograd.Function):
    """The calls of linear's MLP with the cast of its input replaced by the norm, which writes the operand
    of fc1's forward (row-wise) and of its weight gradient (transposed) itself."""

    @staticmethod
    def forward(ctx, x, residual, gamma, eps, w1, b1, w2, b2, c1, c2, pow2: bool):
        ctx.set_materialize_grads(False)
        M, K = x.shape
        H, N = w1.shape[0], w2.shape[0]
        _check_dims(M, K, H, N)
        flags, accum = _fwd_policy(pow2)
        # (the transposed operand is for fc1's weight gradient alone)
        n = te_rmsnorm_fwd(x, gamma, eps, residual=residual, out_dtype=FWD_DTYPE, flags=flags, transpose=ctx.needs_input_grad[4])
        h = x if residual is None else n.h
        qw1, sw1, _, _ = c1.get(w1)
        z1 = torch.empty((M, H), dtype=torch.bfloat16, device=x.device)
        a = te_fp8_gemm_fwd(n.q, n.scales, FWD_DTYPE, qw1, sw1, FWD_DTYPE, bias=b1,
                            epilogue=TE_EPI_BIAS | TE_EPI_GELU | TE_EPI_AUX_PREACT, preact=z1, y_dtype=TE_DTYPE_BF16, accum=accum)
        qa, sa, qat, sat = te_cast_fp8_per_token_transpose(a, FWD_DTYPE, flags)
        qw2, sw2, _, _ = c2.get(w2)
        y = te_fp8_gemm_fwd(qa, sa, FWD_DTYPE, qw2, sw2, FWD_DTYPE, bias=b2, epilogue=TE_EPI_BIAS, y_dtype=TE_DTYPE_BF16,
                            accum=accum)
        mark = x.new_empty(0)    # (as in linear's functions)
        ctx.save_for_backward(h, n.rstd, gamma, n.qt, n.scales_t, z1, qat, sat, w1, w2, mark)
        ctx.c1, ctx.c2, ctx.added, ctx.x_dtype = c1, c2, residual is not None, x.dtype
        return y, (h if residual is not None else None), mark

    @staticmethod
    def backward(ctx, dy, dh_next, _):
        if dy is None:      # only h was used
            return (dh_next.to(ctx.x_dtype) if dh_next is not None else None), dh_next, *[None] * 9
        return _Fp8NormMlpFn.gradients(ctx, dy, dh_next)

    @staticmethod
    @_first_order
    def gradients(ctx, dy, dh_next):
        h, rstd, gamma, qnt, snt, z1, qat, sat, w1, w2, _ = ctx.saved_tensors
        # What is frozen gets no product, no sum, and nothing added to its main_grad.
        need_x, need_res, need_gamma, _, need_w1, need_b1, need_w2, need_b2 = ctx.needs_input_grad[:8]
        through = need_x or need_res or need_gamma      # the gradient goes on below fc1
        d_x = d_res = d_gamma = d_w1 = d_b1 = d_w2 = d_b2 = None
        qdy, sdy, qdyt, sdyt = te_cast_fp8_per_token_transpose(dy.contiguous(), BWD_DTYPE)
        if need_w2 or need_b2:
            w2buf, f2 = _grad_buffer(w2) if need_w2 else (_unread(w2), True)
            db2 = torch.empty((w2.shape[0],), dtype=torch.float32, device=dy.device)
            te_fp8_wgrad_accum_bgrad(qdyt, sdyt, BWD_DTYPE, qat, sat, FWD_DTYPE, w2buf, db2, TE_ACCUM_FULL_FP32)
            d_w2 = None if f2 else w2buf.to(w2.dtype)
            d_b2 = db2.to(torch.bfloat16) if need_b2 else None
        if through or need_w1 or need_b1:
            _, _, qw2t, sw2t = ctx.c2.get(w2)
            db1 = torch.empty((w1.shape[0],), dtype=torch.float32, device=dy.device)
            dz1 = te_fp8_gemm_dgrad_deterministic(qdy, sdy, BWD_DTYPE, qw2t, sw2t, FWD_DTYPE, db1,
                                                  epilogue=TE_EPI_DGELU | TE_EPI_BGRAD, preact=z1, dx_dtype=TE_DTYPE_BF16,
                                                  accum=TE_ACCUM_FULL_FP32)
            d_b1 = db1.to(torch.bfloat16) if need_b1 else None
        if through or need_w1:
            qdz, sdz, qdzt, sdzt = te_cast_fp8_per_token_transpose(dz1, BWD_DTYPE)
        if need_w1:
            w1buf, f1 = _grad_buffer(w1)
            te_fp8_wgrad_accum(qdzt, sdzt, BWD_DTYPE, qnt, snt, FWD_DTYPE, w1buf, TE_ACCUM_FULL_FP32)
            d_w1 = None if f1 else w1buf.to(w1.dtype)
        if through:
            _, _, qw1t, sw1t = ctx.c1.get(w1)
            dn = te_fp8_gemm_dgrad(qdz, sdz, BWD_DTYPE, qw1t, sw1t, FWD_DTYPE, dx_dtype=TE_DTYPE_BF16, accum=TE_ACCUM_FULL_FP32)
            dh, dgamma = te_rmsnorm_bwd(dn, h, rstd, gamma, dres=dh_next.contiguous() if dh_next is not None else None,
                                        need_dgamma=need_gamma)
            d_x, d_res = dh.to(ctx.x_dtype), dh if ctx.added else None
            d_gamma = _to_param(dgamma, gamma) if need_gamma else None
        return d_x, d_res, d_gamma, None, d_w1, d_b1, d_w2, d_b2, None, None, None


class Fp8NormMlp(torch.nn.Module):
    """forward(x, residual=None) -> (mlp(norm(h)), h) with h = x + residual: RmsNorm in front of Fp8Mlp, the
    norm's result going straight into fc1's fp8 operands (from the fp32 value, without the bf16 rounding
    and the cast's pass between the two modules)."""

    def __init__(self, in_features, hidden_features, out_features=None, eps=1e-5, device="cuda", generator=None,
                 pow2_scales=False):
        super().__init__()
        self.norm = RmsNorm(in_features, eps, device)
        self.mlp = Fp8Mlp(in_features, hidden_features, out_features, device=device, generator=generator, pow2_scales=pow2_scales)

    def forward(self, x, residual=None):
        shp, m = x.shape, self.mlp
        flat = residual.reshape(-1, shp[-1]) if residual is not None else None
        y, h, _ = _Fp8NormMlpFn.apply(x.reshape(-1, shp[-1]), flat, self.norm.weight, self.norm.eps, m.w1, m.b1, m.w2, m.b2,
                                      m.c1, m.c2, m.pow2_scales)
        return y.reshape(*shp[:-1], y.shape[-1]), (x if h is None else h.reshape(shp))


class _RouterFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, top_k: int, renormalize: bool, token_mask):
        ctx.set_materialize_grads(False)
        r = te_moe_router_fwd(logits, top_k, renormalize=renormalize, token_mask=token_mask, loss=True)
        ctx.save_for_backward(logits, r.index, r.lse, r.counts, r.routed)
        ctx.renormalize = renormalize
        ctx.mark_non_differentiable(r.index, r.counts)
        return r.weight, r.loss, r.index, r.counts

    @staticmethod
    @_first_order
    def backward(ctx, d_weight, d_loss, _index, _counts):
        logits, index, lse, counts, routed = ctx.saved_tensors
        d = te_moe_router_bwd(logits, index, lse, counts, routed, renormalize=ctx.renormalize,
                              d_weight=d_weight.contiguous() if d_weight is not None else None,
                              d_loss=d_loss.contiguous() if d_loss is not None else None)
        return d, None, None, None


class TopKRouter(torch.nn.Module):
    """forward(logits, token_mask=None) -> (weight, loss, index, counts) of te_moe_router_fwd, with the
    gradients of weight and loss flowing to the logits."""

    def __init__(self, top_k, renormalize=True):
        super().__init__()
        self.top_k, self.renormalize = top_k, renormalize

    def forward(self, logits, token_mask=None):
        return _RouterFn.apply(logits, self.top_k, self.renormalize, token_mask)


def clip_grad_norm(parameters, max_norm):
    """Clips the gradients of the parameters (or of one) in place (main_grad where a parameter has one, else grad) to
    a global norm of at most max_norm and returns the norm, fp32 [1] on the GPU.  Frozen parameters
    (requires_grad False) do not count and are left alone; one that comes several times counts once."""
    parameters = [parameters] if isinstance(parameters, torch.Tensor) else parameters
    trained = {id(p): p for p in parameters if p.requires_grad}.values()
    grads = [getattr(p, "main_grad", None) if getattr(p, "main_grad", None) is not None else p.grad for p in trained]
    return te_grad_norm_clip([g for g in grads if g is not None], max_norm)
