"""Cases of the operators around the FP8 GEMMs in a transformer block's step: the root-mean-square norm with the
residual's addition and its output in 8 bits with scales (forward and backward), the top-k router with its per-expert
counts and balance loss (forward and backward), and the global gradient norm with clipping.

Sizes: 8192 tokens, 4096 and 14336 features, 2112 and 7168 columns, 8 experts and 32768 grouped tokens are those of this
repository's workloads; the rest is generic.
"""
import math

import torch

own = False

EPS = 1e-5            # of the norm
MAX_NORM = 1.0        # of the clipping
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
F8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
SIZE = {"bf16": 2, "f32": 4, "e4m3": 1, "e5m2": 1, "": 0}


def listed():
    return [
        # serving: the norm before a layer for one token (residual stream in bf16, operand of the next GEMM in e4m3)
        dict(name="norm_fwd_1_token", op="norm_fwd", rows=1, cols=4096, x="bf16", h="bf16", out="e4m3", both=False),
        # serving: a ragged batch of tokens at the grouped workload's width, plain bf16 output
        dict(name="norm_fwd_77_tokens", op="norm_fwd", rows=77, cols=7168, x="bf16", h="bf16", out="bf16", both=False),
        # training: the residual added, and the operands of both the forward and the weight gradient in one call
        dict(name="norm_fwd_train", op="norm_fwd", rows=8192, cols=4096, x="bf16", h="bf16", out="e4m3", both=True),
        # a norm of fp32 activations without a residual at a width that is no multiple of 128 and rows that are odd
        dict(name="norm_fwd_f32_2112", op="norm_fwd", rows=4999, cols=2112, x="f32", h="", out="f32", both=False),
        # training: the backward pass with the residual's gradient added
        dict(name="norm_bwd_train", op="norm_bwd", rows=8192, cols=4096, dy="bf16", h="bf16", dres=True),
        # the backward pass of a short batch with an fp32 residual stream
        dict(name="norm_bwd_300", op="norm_bwd", rows=300, cols=2112, dy="bf16", h="f32", dres=True),
        # serving: routing of a few tokens, no loss
        dict(name="router_fwd_4_tokens", op="router_fwd", tokens=4, experts=64, top_k=6, dtype="f32", renorm=True,
             loss=False, closed=0),
        # training: the grouped workload's tokens over its 8 experts
        dict(name="router_fwd_8_experts", op="router_fwd", tokens=32768, experts=8, top_k=2, dtype="f32", renorm=True,
             loss=True, closed=0),
        # training: many experts, some of them closed, bf16 logits (equal logits are common)
        dict(name="router_fwd_256", op="router_fwd", tokens=65536, experts=256, top_k=8, dtype="bf16", renorm=False,
             loss=True, closed=5),
        # training: the backward pass of the same
        dict(name="router_bwd_256", op="router_bwd", tokens=65536, experts=256, top_k=8, dtype="bf16", renorm=False,
             loss=True, closed=5),
        # a small model's gradients: many small tensors, where the launches count
        dict(name="grad_clip_small", op="grad_clip", layers=6, width=192, hidden=500, bias=True, g="f32", out="f32"),
        # the fp32 main gradients of 4 MLP blocks 4096 -> 14336 -> 4096, clipped into the optimizer's bf16 gradients
        dict(name="grad_clip_mlp", op="grad_clip", layers=4, width=4096, hidden=14336, bias=True, g="f32", out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "router_fwd", "router_bwd", "grad_clip"])
    if op == "norm_fwd":
        out = rng.choice(["bf16", "f32", "e4m3", "e5m2"])
        h = rng.choice(["", "bf16", "f32"])
        both = out in F8 and rng.random() < 0.5
        cols = _log(rng, 64, 14336)
        if out in F8:
            cols = max(1, cols // 128) * 128
        elif rng.random() < 0.5:
            cols = max(8, cols // 8 * 8)
        rows = _log(rng, 1, min(16384, 2 ** 24 // cols))
        if both:
            rows = max(1, rows // 128) * 128
        return dict(op=op, rows=rows, cols=cols, x=rng.choice(["bf16", "f32"]), h=h, out=out, both=both)
    if op == "norm_bwd":
        cols = _log(rng, 64, 14336)
        if rng.random() < 0.7:
            cols = max(8, cols // 8 * 8)
        return dict(op=op, rows=_log(rng, 1, min(16384, 2 ** 24 // cols)), cols=cols, dy=rng.choice(["bf16", "f32"]),
                    h=rng.choice(["bf16", "f32"]), dres=rng.random() < 0.7)
    if op in ("router_fwd", "router_bwd"):
        experts = _log(rng, 2, 400)
        return dict(op=op, tokens=_log(rng, 1, min(100000, 2 ** 23 // experts)), experts=experts,
                    top_k=rng.randint(1, min(8, experts)), dtype=rng.choice(["bf16", "f32"]), renorm=rng.random() < 0.5,
                    loss=op == "router_bwd" or rng.random() < 0.7, closed=rng.choice([0, 0, experts // 10]))
    width = _log(rng, 32, 4096)
    return dict(op=op, layers=rng.randint(1, 4), width=width, hidden=_log(rng, width, 3.5 * width), bias=rng.random() < 0.7,
                g=rng.choice(["bf16", "f32"]), out=rng.choice(["bf16", "f32"]))


def _sizes(c):
    """Elements of the gradients of `layers` blocks: norm, fc1, fc2 and their biases."""
    w, h = c["width"], c["hidden"]
    return c["layers"] * ([w, w * h, h, w * h, w] if c["bias"] else [w, w * h, w * h])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(shape, std=1.0, dtype=torch.float32, mean=0.0):
        return torch.randn(shape, generator=gen, device="cuda").mul_(std).add_(mean).to(dtype)

    c, s = case, dict(case=case)
    if c["op"] in ("norm_fwd", "norm_bwd"):
        rows, cols = c["rows"], c["cols"]
        s["gamma"] = normal((cols,), 0.1, torch.bfloat16, 1.0)
        # a residual stream: some channels are far larger than the others
        channel = torch.exp(normal((cols,), 0.5))
        if c["op"] == "norm_fwd":
            s["x"] = normal((rows, cols), 0.7, DT[c["x"]])
            s["res"] = (normal((rows, cols), 1.5) * channel).to(DT[c["h"]]) if c["h"] else None
        else:
            s["h"] = (normal((rows, cols), 1.5) * channel).to(DT[c["h"]])
            s["rstd"] = torch.rsqrt(s["h"].double().square().mean(1) + EPS).float()
            s["dy"] = normal((rows, cols), 1e-3, DT[c["dy"]])
            s["dres"] = normal((rows, cols), 1e-3, DT[c["h"]]) if c["dres"] else None
    elif c["op"] in ("router_fwd", "router_bwd"):
        tokens, experts, k = c["tokens"], c["experts"], c["top_k"]
        # logits with a preference for some experts, as an unbalanced router has; closed experts have none
        logits = normal((tokens, experts)) + normal((experts,), 0.5)
        if c["closed"]:
            logits[:, torch.randperm(experts, generator=gen, device="cuda")[:c["closed"]]] = -math.inf
        s["logits"] = logits.to(DT[c["dtype"]])
        # tokens that only pad the batch are not routed
        s["mask"] = torch.rand((tokens,), generator=gen, device="cuda") < 0.95 if c["loss"] else None
        if c["op"] == "router_bwd":
            out = _plain_router(s["logits"], s["mask"], k, c["renorm"], True)
            s.update({n: out[n] for n in ("index", "lse", "counts", "routed")})
            s["d_weight"] = normal((tokens, k), 1e-3)
            s["d_loss"] = torch.full((1,), 0.01, device="cuda")
    else:
        sizes = _sizes(c)
        # (the tensors of each list lie one after the other in one buffer, as gradient buckets do)
        flat = normal((sum(sizes),), 1e-3, DT[c["g"]])
        s["out"] = torch.empty((sum(sizes),), dtype=DT[c["out"]], device="cuda")
        s["grads"], s["outs"] = list(flat.split(sizes)), list(s["out"].split(sizes))
    return s


# ----------------------------------------------------------------------------------------------- plain forms
def _quantise(y, out):
    """The per-token cast of fp32 y in groups of 128 columns: codes as fp8 values, and scales [cols/128][rows]."""
    dtype, top = F8[out]
    v = y.reshape(y.shape[0], -1, 128)
    amax = v.abs().amax(2).clamp_min(2.0 ** -100)
    q = (v * (top / amax)[..., None]).clamp(-top, top).to(dtype).reshape(y.shape)
    return q, (amax / top).t().contiguous()


def _plain_norm_fwd(s):
    c = s["case"]
    x = s["x"].float()
    h = (x + s["res"].float()).to(s["res"].dtype) if c["h"] else None
    v = h.float() if c["h"] else x
    rstd = torch.rsqrt((v * v).mean(1) + EPS)
    y = v * rstd[:, None] * s["gamma"].float()
    got = dict(h=h, rstd=rstd)
    if c["out"] in F8:
        got["q"], got["scales"] = _quantise(y, c["out"])
        if c["both"]:
            got["qt"], got["scales_t"] = _quantise(y.t().contiguous(), c["out"])
    else:
        got["y"] = y.to(DT[c["out"]])
    return got


def _plain_norm_bwd(s):
    xh = s["h"].float() * s["rstd"][:, None]
    dy = s["dy"].float()
    g = dy * s["gamma"].float()
    dh = s["rstd"][:, None] * (g - xh * (g * xh).mean(1, keepdim=True))
    if s["dres"] is not None:
        dh = dh + s["dres"].float()
    return dict(dh=dh.to(s["h"].dtype), dgamma=(dy * xh).sum(0))


def _plain_router(logits, mask, k, renorm, loss):
    v = logits.float()
    tokens, experts = v.shape
    top = v.amax(1, keepdim=True)
    e = torch.exp(v - top)
    total = e.sum(1, keepdim=True)
    p = e / total
    best, index = torch.sort(v, dim=1, descending=True, stable=True)
    best, index = best[:, :k], index[:, :k]
    chosen = best > -math.inf
    if mask is not None:
        chosen = chosen & mask[:, None]
    w = p.gather(1, index)
    if renorm:
        w = w / (w * (best > -math.inf)).sum(1, keepdim=True)
    got = dict(index=torch.where(chosen, index, -1).to(torch.int32), weight=torch.where(chosen, w, 0.0))
    if loss:
        routed = chosen.any(1)
        n = routed.sum()
        counts = torch.bincount(torch.where(chosen, index, experts).reshape(-1), minlength=experts + 1)[:experts]
        probs = (p * routed[:, None]).sum(0, dtype=torch.float64)
        got["lse"] = torch.where(routed, (top + torch.log(total))[:, 0], 0.0)
        got["counts"], got["routed"] = counts.to(torch.int32), n.to(torch.int32).reshape(1)
        got["loss"] = (experts / k * (counts * probs).sum() / n.clamp_min(1).double().square()).float().reshape(1)
    return got


def _plain_router_bwd(s):
    c = s["case"]
    k, experts = c["top_k"], c["experts"]
    index, n = s["index"], s["routed"].clamp_min(1).float()
    routed = index[:, :1] >= 0
    p = torch.where(routed, torch.exp(s["logits"].float() - s["lse"][:, None]), 0.0)
    a = s["d_loss"] * (experts / k) * s["counts"].float() / (n * n)
    chosen = index >= 0
    at = index.clamp_min(0).long()
    dw = torch.where(chosen, s["d_weight"], 0.0)
    if c["renorm"]:
        w = torch.where(chosen, p.gather(1, at), 0.0)
        w = w / w.sum(1, keepdim=True).clamp_min(1e-30)
        d = p * (a - (p * a).sum(1, keepdim=True))
        d = d.scatter_add(1, at, w * (dw - (w * dw).sum(1, keepdim=True)))
    else:
        b = a.expand_as(p).scatter_add(1, at, dw)
        d = p * (b - (p * b).sum(1, keepdim=True))
    return dict(d_logits=d.to(s["logits"].dtype))


def _plain_clip(s):
    total = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]]).sum()
    norm = total.sqrt().float()
    coef = (MAX_NORM / (norm + 1e-6)).clamp_max(1.0)
    [o.copy_(g.float() * coef) for o, g in zip(s["outs"], s["grads"])]
    return dict(norm=norm.reshape(1), out=s["out"])


# --------------------------------------------------------------------------------------------- the framework's
def _own(s):
    import fp8_linear_layer_amd as te
    c = s["case"]
    if c["op"] == "norm_fwd":
        fp8 = c["out"] in F8
        r = te.te_rmsnorm_fwd(s["x"], s["gamma"], EPS, residual=s["res"],
                              out_dtype=dict(bf16=te.TE_DTYPE_BF16, f32=te.TE_DTYPE_F32, e4m3=te.TE_DTYPE_E4M3,
                                             e5m2=te.TE_DTYPE_E5M2)[c["out"]], transpose=c["both"])
        got = dict(h=r.h, rstd=r.rstd)
        if fp8:
            got["q"], got["scales"] = r.q.view(F8[c["out"]][0]), r.scales[:, :c["rows"]]
            if c["both"]:
                got["qt"], got["scales_t"] = r.qt.view(F8[c["out"]][0]), r.scales_t[:, :c["cols"]]
        else:
            got["y"] = r.y
        return got
    if c["op"] == "norm_bwd":
        dh, dgamma = te.te_rmsnorm_bwd(s["dy"], s["h"], s["rstd"], s["gamma"], dres=s["dres"])
        return dict(dh=dh, dgamma=dgamma)
    if c["op"] == "router_fwd":
        r = te.te_moe_router_fwd(s["logits"], c["top_k"], renormalize=c["renorm"], token_mask=s["mask"], loss=c["loss"])
        got = dict(index=r.index, weight=r.weight)
        if c["loss"]:
            got.update(lse=r.lse, counts=r.counts, routed=r.routed, loss=r.loss)
        return got
    if c["op"] == "router_bwd":
        return dict(d_logits=te.te_moe_router_bwd(s["logits"], s["index"], s["lse"], s["counts"], s["routed"],
                                                  d_weight=s["d_weight"], d_loss=s["d_loss"], renormalize=c["renorm"]))
    return dict(norm=te.te_grad_norm_clip(s["grads"], MAX_NORM, out=s["outs"]), out=s["out"])


def run(state):
    if own:
        return _own(state)
    c = state["case"]
    if c["op"] == "norm_fwd":
        return _plain_norm_fwd(state)
    if c["op"] == "norm_bwd":
        return _plain_norm_bwd(state)
    if c["op"] == "router_fwd":
        return _plain_router(state["logits"], state["mask"], c["top_k"], c["renorm"], c["loss"])
    if c["op"] == "router_bwd":
        return _plain_router_bwd(state)
    return _plain_clip(state)


def work(case):
    c = case
    if c["op"] == "norm_fwd":
        n = c["rows"] * c["cols"]
        b = n * (SIZE[c["x"]] + 2 * SIZE[c["h"]] + SIZE[c["out"]] * (2 if c["both"] else 1)) + 2 * c["cols"] + 4 * c["rows"]
        b += (n // 128 * 4) * (2 if c["both"] else 1) if c["out"] in F8 else 0
        return dict(bytes=b, flops=6 * n)
    if c["op"] == "norm_bwd":
        n = c["rows"] * c["cols"]
        return dict(bytes=n * (SIZE[c["dy"]] + SIZE[c["h"]] * (3 if c["dres"] else 2)) + 6 * c["cols"] + 4 * c["rows"],
                    flops=12 * n)
    if c["op"] == "router_fwd":
        n, t = c["tokens"] * c["experts"], c["tokens"]
        return dict(bytes=n * SIZE[c["dtype"]] + t * c["top_k"] * 8 + ((5 * t + 4 * c["experts"]) if c["loss"] else 0),
                    flops=(5 + c["top_k"]) * n)
    if c["op"] == "router_bwd":
        n, t = c["tokens"] * c["experts"], c["tokens"]
        return dict(bytes=2 * n * SIZE[c["dtype"]] + t * c["top_k"] * 8 + 4 * t + 4 * c["experts"], flops=8 * n)
    n = sum(_sizes(c))
    return dict(bytes=n * (SIZE[c["g"]] + SIZE[c["out"]]), flops=3 * n)


# ------------------------------------------------------------------------------------------------ 64-bit values
def _exact_cast(y, top):
    groups = y.unflatten(1, (-1, 128))
    amax = groups.abs().amax(-1)
    return (groups / amax.unsqueeze(-1) * top).flatten(1), (amax / top).transpose(0, 1)


def _exact_norm_fwd(s, c):
    v = s["x"].double()
    got = {}
    if c["h"]:
        got["h"] = v + s["res"].double()
        # (the stored sum, in its own type, is what the norm is of)
        v = got["h"].float().to(DT[c["h"]]).double()
    ms = torch.linalg.vector_norm(v, dim=1).pow(2) / c["cols"]
    got["rstd"] = 1.0 / torch.sqrt(ms + EPS)
    y = torch.einsum("rc,r,c->rc", v, got["rstd"], s["gamma"].double())
    if c["out"] not in F8:
        got["y"] = y
        return got
    got["q"], got["scales"] = _exact_cast(y, F8[c["out"]][1])
    if c["both"]:
        got["qt"], got["scales_t"] = _exact_cast(y.transpose(0, 1), F8[c["out"]][1])
    return got


def _exact_norm_bwd(s, c):
    # the gradient by differentiation of the norm as a function of its row, with the given 1/rms as its value
    h, r, dy = s["h"].double(), s["rstd"].double().unsqueeze(1), s["dy"].double()
    through = torch.einsum("rc,c->rc", dy, s["gamma"].double())
    along = torch.einsum("rc,rc->r", through, h).unsqueeze(1) * r.pow(3) / c["cols"]
    dh = r * through - along * h
    if s["dres"] is not None:
        dh += s["dres"].double()
    return dict(dh=dh, dgamma=torch.einsum("rc,rc,r->c", dy, h, r.squeeze(1)))


def _exact_router(s, c):
    v, k = s["logits"].double(), c["top_k"]
    tokens, experts = v.shape
    p = torch.softmax(v, 1)
    order = torch.argsort(-v, dim=1, stable=True)[:, :k]
    usable = torch.isfinite(torch.gather(v, 1, order))
    if s["mask"] is not None:
        usable &= s["mask"].unsqueeze(1)
    w = torch.where(usable, torch.gather(p, 1, order), 0.0)
    if c["renorm"]:
        w = w / torch.where(usable, w, 0.0).sum(1, keepdim=True).clamp_min(1e-300)
    got = dict(index=order.masked_fill(~usable, -1).to(torch.int32), weight=w)
    if c["loss"]:
        live = usable[:, 0]
        n = int(live.sum())
        hits = torch.zeros((tokens, experts), dtype=torch.float64, device=v.device).scatter_(1, order, usable.double())
        got["counts"] = hits.sum(0).round().to(torch.int32)
        got["routed"] = torch.tensor([n], dtype=torch.int32)
        got["lse"] = torch.logsumexp(v, 1).masked_fill(~live, 0.0)
        share, mean = hits.sum(0) / max(1, n * k), p[live].sum(0) / max(1, n)
        got["loss"] = (experts * (share * mean).sum()).reshape(1)
    return got


def _exact_router_bwd(s, c):
    v, k, n = s["logits"].double(), c["top_k"], max(1, int(s["routed"]))
    index = s["index"].long()
    live = index[:, 0] >= 0
    v = torch.where(live.unsqueeze(1), v, 0.0).requires_grad_()
    p = torch.softmax(v, 1)
    picked = torch.where(index >= 0, p.gather(1, index.clamp(min=0)), 0.0)
    if c["renorm"]:
        picked = picked / picked.sum(1, keepdim=True).clamp_min(1e-300)
    value = (picked * s["d_weight"].double()).sum()
    share = s["counts"].double() / (n * k)
    value = value + s["d_loss"].double()[0] * c["experts"] * (p[live].sum(0) / n * share).sum()
    value.backward()
    return dict(d_logits=v.grad.masked_fill(~live.unsqueeze(1), 0.0))


def _exact_clip(s):
    norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(g, dtype=torch.float64)) ** 2 for g in s["grads"]))
    coef = min(1.0, MAX_NORM / (norm + 1e-6))
    return dict(norm=torch.tensor([norm], dtype=torch.float64), out=torch.cat([g.double() * coef for g in s["grads"]]))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_fwd":
        return _exact_norm_fwd(s, case)
    if case["op"] == "norm_bwd":
        return _exact_norm_bwd(s, case)
    if case["op"] == "router_fwd":
        return _exact_router(s, case)
    if case["op"] == "router_bwd":
        return _exact_router_bwd(s, case)
    return _exact_clip(s)
