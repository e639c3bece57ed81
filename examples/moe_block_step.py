"""Training steps of a small mixture-of-experts block on the library: a norm in front of an FP8 MLP, a
second norm, the router, the experts' FP8 products over the routed tokens, and the gradients clipped.

  h1 = x0 (+ nothing);        y1 = mlp(norm(h1))                      Fp8NormMlp
  h2 = y1 + h1;               y2 = norm(h2)                           RmsNorm
  weight, loss, index, counts = router(y2 Wr)                         TopKRouter
  out = h2 + sum over a token's experts of weight * (We y2)           M-grouped GEMM, K-grouped weight gradient
  step: backward, clip_grad_norm over the fp32 gradients, plain gradient descent

Tokens are dealt out without a copy to the host: every expert's rows start at a multiple of 256 (the
M-grouped layout), in a buffer that is large enough for any counts.

    python examples/moe_block_step.py [--tokens 2048] [--width 512] [--hidden 1024] [--experts 8] [--steps 10]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_linear_layer_amd as te  # noqa: E402
from fp8_linear_layer_amd.block import Fp8NormMlp, RmsNorm, TopKRouter, clip_grad_norm  # noqa: E402

E4, E5 = te.TE_DTYPE_E4M3, te.TE_DTYPE_E5M2
BLOCK = 256


def deal(index, counts, experts):
    """Where each (token, choice) goes: its row in the experts' buffer, the expert of each 256-row block of
    the buffer (-1: unused) and the rows of each expert, padded to whole blocks."""
    tokens, k = index.shape
    rows = (tokens * k + experts * (BLOCK - 1) + BLOCK - 1) // BLOCK * BLOCK
    padded = (counts.long() + BLOCK - 1) // BLOCK * BLOCK
    end = padded.cumsum(0)
    flat = index.reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    expert = flat[order]                                    # (-1 first: tokens that go nowhere)
    first = torch.searchsorted(expert, expert)              # first entry of the same expert
    place = torch.arange(tokens * k, device=index.device) - first
    row = torch.where(expert >= 0, (end - padded)[expert.clamp_min(0)] + place, rows)
    where = torch.empty_like(flat)
    where[order] = row
    block = torch.arange(0, rows, BLOCK, device=index.device)
    owner = torch.searchsorted(end, block, right=True)
    owner = torch.where(owner < experts, owner, -1).int()
    return where.reshape(tokens, k), owner, padded, rows


class _Experts(torch.autograd.Function):
    """rows = the tokens' vectors dealt to the experts' buffer; out[row] = W[expert of the row] rows[row]."""

    @staticmethod
    def forward(ctx, rows, w, owner, padded):
        q, s, qt, st = te.te_cast_fp8_per_token_transpose(rows, E4)
        experts, n, k = w.shape
        qw = torch.empty((experts, n, k), dtype=torch.uint8, device=w.device)
        sw = torch.empty((experts, k // 128, te.scale_ld(n)), dtype=torch.float32, device=w.device)
        qwt = torch.empty((experts, k, n), dtype=torch.uint8, device=w.device)
        swt = torch.empty((experts, n // 128, te.scale_ld(k)), dtype=torch.float32, device=w.device)
        for e in range(experts):
            te.te_cast_fp8_per_token_transpose(w[e].detach(), E4, q=qw[e], scales=sw[e], qt=qwt[e], scales_t=swt[e])
        y = torch.zeros((rows.shape[0], n), dtype=torch.bfloat16, device=rows.device)      # (unused blocks are not written)
        te.te_fp8_mgrouped_gemm_fwd(q, s, E4, qw, sw, E4, owner, y=y, accum=te.TE_ACCUM_FULL_FP32)
        ctx.save_for_backward(qt, st, qwt, swt, owner, padded)
        ctx.w = w
        return y

    @staticmethod
    def backward(ctx, dy):
        qt, st, qwt, swt, owner, padded = ctx.saved_tensors
        qd, sd, qdt, sdt = te.te_cast_fp8_per_token_transpose(dy.contiguous(), E5)
        dx = torch.zeros((dy.shape[0], qwt.shape[1]), dtype=torch.bfloat16, device=dy.device)
        te.te_fp8_mgrouped_gemm_dgrad(qd, sd, E5, qwt, swt, E4, owner, dx=dx)
        te.te_fp8_kgrouped_wgrad_device_sizes(qdt, sdt, E5, qt, st, E4, padded, ctx.w.main_grad)
        return dx, None, None, None


class MoeBlock(torch.nn.Module):
    def __init__(self, width, hidden, experts, top_k, generator):
        super().__init__()
        self.dense = Fp8NormMlp(width, hidden, generator=generator)
        self.norm = RmsNorm(width)
        self.gate = torch.nn.Parameter((torch.randn(experts, width, generator=generator, device="cuda") / width ** 0.5).bfloat16())
        self.router = TopKRouter(top_k)
        self.experts = torch.nn.Parameter(
            (torch.randn(experts, width, width, generator=generator, device="cuda") / width ** 0.5).bfloat16())
        self.experts.main_grad = torch.zeros(self.experts.shape, dtype=torch.float32, device="cuda")

    def forward(self, x, token_mask=None):
        y, h = self.dense(x)
        y, h = self.norm(y, h)
        weight, loss, index, counts = self.router(torch.nn.functional.linear(y, self.gate), token_mask)
        where, owner, padded, n = deal(index, counts, self.experts.shape[0])
        token = torch.arange(x.shape[0], device=x.device)[:, None].expand_as(where)
        rows = torch.zeros((n + 1, x.shape[1]), dtype=torch.bfloat16, device=x.device).index_copy(
            0, where.reshape(-1), y[token.reshape(-1)])[:n]
        out = _Experts.apply(rows, self.experts, owner, padded)
        picked = torch.cat([out, out.new_zeros((1, out.shape[1]))])[where.reshape(-1)].reshape(*where.shape, -1)
        return h + (picked * weight[..., None]).sum(1).to(h.dtype), loss, counts


def main(argv=None):
    ap = argparse.ArgumentParser()
    for name, value in (("tokens", 2048), ("width", 512), ("hidden", 1024), ("experts", 8), ("top-k", 2), ("steps", 10)):
        ap.add_argument(f"--{name}", type=int, default=value)
    ap.add_argument("--lr", type=float, default=4.0)
    ap.add_argument("--balance", type=float, default=0.01)
    ap.add_argument("--max-norm", type=float, default=0.15)
    a = ap.parse_args(argv)
    gen = torch.Generator(device="cuda").manual_seed(0)
    block = MoeBlock(a.width, a.hidden, a.experts, a.top_k, gen)
    x = torch.randn(a.tokens, a.width, generator=gen, device="cuda").bfloat16()
    goal = torch.randn(a.tokens, a.width, generator=gen, device="cuda").bfloat16() * 0.5 + x
    mask = torch.arange(a.tokens, device="cuda") % 37 != 0          # some tokens only pad the batch
    history = []
    for step in range(a.steps):
        out, balance, counts = block(x, mask)
        task = ((out.float() - goal.float()) ** 2).mean()
        (task + a.balance * balance[0]).backward()
        norm = clip_grad_norm(block.parameters(), a.max_norm)
        with torch.no_grad():
            for p in block.parameters():
                g = getattr(p, "main_grad", None)
                p.sub_((a.lr * (g if g is not None else p.grad)).to(p.dtype))
                p.grad = None
                if g is not None:
                    g.zero_()
        history.append((float(task.detach()), float(balance.detach()), float(norm)))
        print(f"step {step}: loss {history[-1][0]:.4f} balance {history[-1][1]:.4f} gradient norm {history[-1][2]:.4f} "
              f"tokens per expert {counts.tolist()}", flush=True)
    return history


if __name__ == "__main__":
    main()
