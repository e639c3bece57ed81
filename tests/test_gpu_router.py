"""GPU parity of te_moe_router_fwd / te_moe_router_bwd with the formulas in 64 bits.

Choices and counts have to be equal.  Tolerances (u = 2^-24): with x = logit - largest, exp(x) is off by
x's rounding and the exponent's, together 4 |x| u, and a few u of its own; the sum of the row weighs
those by the terms themselves, so 128 u covers it with its additions, and a weight is within
(128 + 4 |x|) u.  The loss and the column sums have positive terms of that accuracy."""
import math

import pytest
import torch

te = pytest.importorskip("fp8_linear_layer_amd")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
INF, NAN = float("inf"), float("nan")
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    te.load_library()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def make_logits(tokens, experts, dtype, seed, closed=0, ld=None, shift=0, std=1.0):
    g = gen(seed)
    ld = ld or experts
    buf = torch.full((tokens * ld + shift + 8,), NAN, dtype=dtype, device="cuda")
    v = buf[shift:].as_strided((tokens, experts), (ld, 1))
    v.copy_(torch.randn((tokens, experts), generator=g, device="cuda") * std +
            torch.randn((experts,), generator=g, device="cuda") * 0.5)
    if closed:
        v[:, torch.randperm(experts, generator=g, device="cuda")[:closed]] = -INF
    return v


def exact(logits, k, renorm, mask=None):
    v = logits.double()
    tokens, experts = v.shape
    best, order = torch.sort(v, dim=1, descending=True, stable=True)
    best, order = best[:, :k], order[:, :k]
    ok = best > -INF
    if mask is not None:
        ok &= mask.bool()[:, None]
    top = torch.where(ok[:, :1], best[:, :1], 0.0)
    total = (v - top).exp().sum(1, keepdim=True)
    lse = (top + total.log())[:, 0]
    w = torch.where(ok, (best - top).exp() / total, 0.0)      # (not through lse, which may be too large to hold log(total))
    if renorm:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    live = ok[:, 0]
    n = int(live.sum())
    counts = torch.bincount(order[ok], minlength=experts)
    p = torch.where(live[:, None], (v - top).exp() / total, 0.0)
    loss = experts / k * float((counts.double() * p.sum(0)).sum()) / max(n, 1) ** 2
    return dict(index=torch.where(ok, order, -1).int(), weight=w, lse=torch.where(live, lse, 0.0), x=torch.where(ok, top - best, 0.0),
                counts=counts.int(), n=n, loss=loss, live=live, p=p)


def check_fwd(r, e, loss=True):
    assert torch.equal(r.index, e["index"])
    assert ((r.weight.double() - e["weight"]).abs() <= (128 + 4 * e["x"]) * U * e["weight"]).all()
    if r.lse is not None:
        assert ((r.lse.double() - e["lse"]).abs() <= 128 * U + 4 * U * e["lse"].abs()).all()
    if loss:
        assert torch.equal(r.counts, e["counts"]) and int(r.routed) == e["n"]
        assert abs(float(r.loss) - e["loss"]) <= 256 * U * e["loss"]


EXPERTS = [1, 2, 3, 7, 8, 9, 12, 16, 17, 31, 32, 33, 40, 64, 65, 77, 128, 129, 200, 256, 257, 400, 511, 512, 513, 1000, 1024, 1025, 2048]


@pytest.mark.parametrize("experts", EXPERTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forward(experts, dtype):
    for tokens, k, renorm in ((1, 1, False), (3, 2, True), (67, 3, False), (133, 6, True), (700, 8, False), (40, 16, True), (5000, 4, True)):
        k = min(k, experts)
        closed = experts // 10
        v = make_logits(tokens, experts, DT[dtype], experts * 3 + tokens, closed)
        mask = torch.rand((tokens,), generator=gen(tokens), device="cuda") < 0.8
        r = te.te_moe_router_fwd(v, k, renormalize=renorm, token_mask=mask, loss=True)
        check_fwd(r, exact(v, k, renorm, mask))
        assert r.index.dtype == torch.int32 and r.weight.dtype == torch.float32
        s = te.te_moe_router_fwd(v, k, renormalize=renorm)      # serving: no mask, no loss
        check_fwd(s, exact(v, k, renorm), loss=False)
        assert s.lse is None and s.counts is None and s.routed is None and s.loss is None
        again = te.te_moe_router_fwd(v, k, renormalize=renorm, token_mask=mask, loss=True)
        assert all(torch.equal(a, b) for a, b in zip(r, again))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("experts,k", [(6, 4), (16, 8), (64, 8), (100, 7), (256, 8), (300, 16), (2048, 16)])
def test_equal_logits_go_to_the_lower_expert(dtype, experts, k):
    g = gen(experts)
    v = torch.randint(-2, 3, (500, experts), generator=g, device="cuda").to(DT[dtype])
    v[0] = 0.0
    v[1] = -0.0
    v[2] = torch.where(torch.arange(experts, device="cuda") % 2 == 0, -0.0, 0.0)     # equal zeros of both signs
    v[3] = -3e38
    check_fwd(te.te_moe_router_fwd(v, k, loss=True), exact(v, k, False))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("experts", [5, 13, 60, 250, 333, 1024])
def test_empty_rows_and_few_open_experts(dtype, experts):
    k = min(4, experts)
    v = make_logits(300, experts, DT[dtype], experts, std=4.0)
    v[::7] = -INF                       # no expert is open
    v[1::7, 2:] = -INF                  # two are
    v[2::7, 1:] = torch.finfo(DT[dtype]).min     # the type's lowest value is a logit, not a closed expert
    v[3::7] = torch.finfo(DT[dtype]).min
    for mask in (None, torch.zeros((300,), dtype=torch.bool, device="cuda"), torch.arange(300, device="cuda") % 3 == 0):
        for renorm in (False, True):
            r = te.te_moe_router_fwd(v, k, renormalize=renorm, token_mask=mask, loss=True)
            check_fwd(r, exact(v, k, renorm, mask))
            assert (r.index[::7] == -1).all() and (r.weight[::7] == 0).all() and (r.lse[::7] == 0).all()
            dw = torch.ones_like(r.weight)
            d = te.te_moe_router_bwd(v, r.index, r.lse, r.counts, r.routed, d_weight=dw, d_loss=torch.ones(1, device="cuda"),
                                     renormalize=renorm)
            assert (d[r.index[:, 0] < 0] == 0).all()
            check_bwd(v, r, k, renorm, d, dw, torch.ones(1, device="cuda"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("experts", [6, 50, 256, 700])
def test_nan_and_infinite_logits(dtype, experts):
    k = 3
    v = make_logits(64, experts, DT[dtype], experts)
    clean = v.clone()
    neg_nan = torch.tensor(-1, dtype=torch.int16 if dtype == "bf16" else torch.int32, device="cuda").view(DT[dtype])
    v[5, 1], v[9, 4], v[11, experts - 1] = NAN, neg_nan, INF
    v[13] = NAN
    mask = torch.ones((64,), dtype=torch.bool, device="cuda")
    mask[[5, 9, 11, 13]] = False
    r = te.te_moe_router_fwd(v, k, token_mask=mask, loss=True)      # masked tokens do not reach the loss
    check_fwd(r, exact(clean, k, False, mask))
    for renorm in (False, True):
        s = te.te_moe_router_fwd(v, k, renormalize=renorm, loss=True)
        bad = ~mask
        bad[13] = False
        assert s.weight[bad].isnan().all() and s.lse[bad].isnan().all() and s.loss.isnan()
        # no NaN is chosen, the others in their order
        want = exact(torch.where(v.isnan(), -INF, v), k, False)["index"]
        assert torch.equal(s.index, want)
        assert (s.index[13] == -1).all() and (s.weight[13] == 0).all() and s.lse[13] == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("experts,ld,shift", [(9, 11, 1), (64, 67, 1), (77, 77, 3), (256, 261, 5), (6, 7, 1)])
def test_strides_and_alignment(dtype, experts, ld, shift):
    tokens, k = 210, 3
    v = make_logits(tokens, experts, DT[dtype], 5, ld=ld, shift=shift)
    r = te.te_moe_router_fwd(v, k, loss=True)
    e = exact(v, k, False)
    check_fwd(r, e)
    buf = torch.full((tokens * (ld + 1) + 16,), 7.0, dtype=DT[dtype], device="cuda")
    d = buf[shift:].as_strided((tokens, experts), (ld + 1, 1))
    dw = torch.randn((tokens, k), generator=gen(1), device="cuda")
    args = dict(d_weight=dw, d_loss=torch.full((1,), 0.5, device="cuda"))
    te.te_moe_router_bwd(v, r.index, r.lse, r.counts, r.routed, d_logits=d, **args)
    check_bwd(v, r, k, False, d, **args)
    d.fill_(7.0)
    assert (buf == 7.0).all()


# ------------------------------------------------------------ backward
def exact_bwd(v, r, k, renorm, d_weight, d_loss):
    """The gradient and the sum of its terms' magnitudes."""
    x = v.double()
    tokens, experts = x.shape
    index = r.index.long()
    ok = index >= 0
    live = ok[:, :1]
    p = torch.where(live, torch.softmax(x, 1), 0.0)
    a = torch.zeros((experts,), dtype=torch.float64, device=v.device)
    if d_loss is not None:
        n = max(int(r.routed), 1)
        a = float(d_loss) * experts / k * r.counts.double() / (n * n)
    a = a.expand(tokens, experts)
    dw = torch.where(ok, d_weight.double(), 0.0) if d_weight is not None else torch.zeros(index.shape, dtype=torch.float64, device=v.device)
    at = index.clamp_min(0)
    if renorm:
        w = torch.where(ok, p.gather(1, at), 0.0)
        w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
        d = p * (a - (p * a).sum(1, keepdim=True))
        mag = p * (a.abs() + (p * a.abs()).sum(1, keepdim=True))
        d = d.scatter_add(1, at, w * (dw - (w * dw).sum(1, keepdim=True)))
        mag = mag.scatter_add(1, at, w * (dw.abs() + (w * dw.abs()).sum(1, keepdim=True)))
    else:
        b = a.scatter_add(1, at, dw)
        d = p * (b - (p * b).sum(1, keepdim=True))
        b = a.abs().scatter_add(1, at, dw.abs())
        mag = p * (b + (p * b).sum(1, keepdim=True))
    far = torch.where(live, (x - r.lse.double()[:, None]).abs().clamp_max(200.0), 0.0)
    return d, mag * (128 + 4 * far)


def check_bwd(v, r, k, renorm, got, d_weight=None, d_loss=None):
    want, mag = exact_bwd(v, r, k, renorm, d_weight, d_loss)
    err = (got.double() - want).abs()
    # (results below the smallest normal number of the type: half a step there)
    assert (err <= U * mag + HALF[got.dtype] * want.abs() + 2.0 ** -133).all(), float((err / (U * mag + 1e-300)).max())


@pytest.mark.parametrize("experts", EXPERTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward(experts, dtype):
    for tokens, k, renorm in ((1, 1, False), (3, 2, True), (67, 3, False), (133, 6, True), (700, 8, False), (40, 16, True), (9000, 4, True)):
        k = min(k, experts)
        v = make_logits(tokens, experts, DT[dtype], experts * 3 + tokens, experts // 10)
        mask = torch.rand((tokens,), generator=gen(tokens), device="cuda") < 0.8
        r = te.te_moe_router_fwd(v, k, renormalize=renorm, token_mask=mask, loss=True)
        dw = torch.randn((tokens, k), generator=gen(9), device="cuda")
        dl = torch.full((1,), 0.25, device="cuda")
        for args in (dict(d_weight=dw, d_loss=dl), dict(d_weight=dw), dict(d_loss=dl), dict()):
            d = te.te_moe_router_bwd(v, r.index, r.lse, r.counts, r.routed, renormalize=renorm, **args)
            check_bwd(v, r, k, renorm, d, **args)
        assert (d == 0).all()      # neither gradient
        a = te.te_moe_router_bwd(v, r.index, r.lse, r.counts, r.routed, renormalize=renorm, d_weight=dw, d_loss=dl)
        b = te.te_moe_router_bwd(v, r.index, r.lse, r.counts, r.routed, renormalize=renorm, d_weight=dw, d_loss=dl)
        assert torch.equal(a, b)


@pytest.mark.parametrize("renorm", [False, True])
def test_backward_against_differences(renorm):
    """The derivative of sum(weight * dw) + dl * loss along a direction that leaves the choice of experts as
    it is, from the forward kernel's outputs at logits +- step * d.  Their rounding adds at most 160 u of the
    terms / step (the loss 256 u); the differences' own error is that of the same differences in 64 bits."""
    tokens, experts, k, step = 24, 40, 4, 2.0 ** -7
    g = gen(2)
    v = torch.randperm(experts, generator=g, device="cuda").float().expand(tokens, experts).clone() / 8
    v = v[:, torch.randperm(experts, generator=g, device="cuda")] + torch.arange(tokens, device="cuda")[:, None] / 64
    d = torch.randint(-2, 3, (tokens, experts), generator=g, device="cuda").float()      # |step * d| < half the gaps
    dw = torch.randn((tokens, k), generator=g, device="cuda")
    dl = torch.full((1,), 0.7, device="cuda")
    r = te.te_moe_router_fwd(v, k, renormalize=renorm, loss=True)
    grad = te.te_moe_router_bwd(v, r.index, r.lse, r.counts, r.routed, d_weight=dw, d_loss=dl, renormalize=renorm)

    def value(at, kernel):
        if kernel:
            s = te.te_moe_router_fwd(at, k, renormalize=renorm, loss=True)
            assert torch.equal(s.index, r.index)
            return float((s.weight.double() * dw.double()).sum()) + 0.7 * float(s.loss)
        e = exact(at, k, renorm)
        return float((e["weight"] * dw.double()).sum()) + 0.7 * e["loss"]

    diff, diff64 = ((value(v + step * d, kern) - value(v - step * d, kern)) / (2 * step) for kern in (True, False))
    want, mag = exact_bwd(v, r, k, renorm, dw, dl)
    along = float((grad.double() * d.double()).sum())
    terms = float((r.weight.double() * dw.double().abs()).sum())
    tol = (160 * U * terms + 256 * U * 0.7 * float(r.loss)) / step
    tol += abs(diff64 - float((want * d.double()).sum()))
    tol += float(((U * mag + U * want.abs()) * d.double().abs()).sum())
    # (0.7 in fp32)
    tol += U * abs(diff)
    assert abs(along - diff) <= tol, (along, diff, tol)


# ------------------------------------------------------------ both
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_tokens(dtype):
    v = torch.empty((0, 12), dtype=DT[dtype], device="cuda")
    r = te.te_moe_router_fwd(v, 2, loss=True)
    assert r.index.shape == (0, 2) and (r.counts == 0).all() and int(r.routed) == 0 and float(r.loss) == 0
    assert te.te_moe_router_fwd(v, 2).weight.shape == (0, 2)
    d = te.te_moe_router_bwd(v, r.index, r.lse, r.counts, r.routed, d_loss=torch.ones(1, device="cuda"))
    assert d.shape == (0, 12)


def test_indices_outside_the_experts_are_ignored():
    v = make_logits(50, 20, torch.float32, 4)
    r = te.te_moe_router_fwd(v, 3, loss=True)
    dw = torch.randn((50, 3), generator=gen(1), device="cuda")
    wild = r.index.clone()
    wild[:, 2] = 1 << 30
    masked = r.index.clone()
    masked[:, 2] = -1
    a = te.te_moe_router_bwd(v, wild, r.lse, d_weight=dw, renormalize=True)
    b = te.te_moe_router_bwd(v, masked, r.lse, d_weight=dw, renormalize=True)
    assert torch.equal(a, b)


def test_offsets_past_32_bits():
    tokens, experts, ld = 3, 70, 1 << 31
    big = torch.empty((2 * ld + experts,), dtype=torch.bfloat16, device="cuda")
    v = big.as_strided((tokens, experts), (ld, 1))
    small = make_logits(tokens, experts, torch.bfloat16, 8)
    v.copy_(small)
    a, b = te.te_moe_router_fwd(v, 4, loss=True), te.te_moe_router_fwd(small, 4, loss=True)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    dw = torch.ones((tokens, 4), device="cuda")
    da, db = (te.te_moe_router_bwd(t, a.index, a.lse, d_weight=dw) for t in (v, small))
    assert torch.equal(da, db)


def test_given_stream():
    v = make_logits(5000, 40, torch.float32, 6)
    want = te.te_moe_router_fwd(v, 4, loss=True)
    dw = torch.ones((5000, 4), device="cuda")
    dwant = te.te_moe_router_bwd(v, want.index, want.lse, d_weight=dw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = te.te_moe_router_fwd(v, 4, loss=True, stream=side)
    dgot = te.te_moe_router_bwd(v, got.index, got.lse, d_weight=dw, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and torch.equal(dwant, dgot)


def test_other_stream_and_graph():
    tokens, experts, k = 3000, 48, 4
    v = make_logits(tokens, experts, torch.bfloat16, 6)
    dw = torch.randn((tokens, k), generator=gen(1), device="cuda")
    dl = torch.full((1,), 0.01, device="cuda")

    def step():
        r = te.te_moe_router_fwd(v, k, loss=True)
        return [*r, te.te_moe_router_bwd(v, r.index, r.lse, r.counts, r.routed, d_weight=dw, d_loss=dl)]

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        v.copy_(torch.randn((tokens, experts), generator=gen(50 + i), device="cuda"))
        graph.replay()
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager)), i
    assert math.isfinite(float(out[5]))
