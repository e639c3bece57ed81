"""The modules' own logic (block.py, linear.py) on the CPU, with torch in the place of the library's calls: which
gradients a backward pass computes and accumulates, and what clip_grad_norm takes.

The stand-ins keep the calls' signatures and layouts and leave out the 8-bit rounding, so that gradients can be
compared with autograd's (bf16 stores: a few half steps of 2^-8)."""
import math

import pytest
import torch

te = pytest.importorskip("fp8_linear_layer_amd")
from fp8_linear_layer_amd import block, linear  # noqa: E402
from fp8_linear_layer_amd.ops import RmsNormOutput, RouterOutput  # noqa: E402


class Calls:
    """The library's calls in torch; `log` has their names, `options` what a call was asked for beside its operands."""

    def __init__(self):
        self.log, self.options = [], []

    def said(self, name, **options):
        self.log.append(name)
        self.options.append(dict(name=name, **options))

    def te_rmsnorm_fwd(self, x, gamma, eps=1e-5, residual=None, out_dtype=te.TE_DTYPE_BF16, flags=0, transpose=False):
        self.said("norm", transpose=transpose)
        h = (x.float() + residual.float()).to(residual.dtype) if residual is not None else None
        v = (h if h is not None else x).float()
        rstd = torch.rsqrt((v * v).mean(1) + eps)
        y = v * rstd[:, None] * gamma.float()
        fp8 = out_dtype not in (te.TE_DTYPE_BF16, te.TE_DTYPE_F32)
        return RmsNormOutput(h, rstd, None if fp8 else y.bfloat16(), y if fp8 else None, None,
                             y.t().contiguous() if transpose else None, None)

    def te_rmsnorm_bwd(self, dy, h, rstd, gamma, dres=None, need_dgamma=True):
        self.said("norm_bwd", need_dgamma=need_dgamma)
        xh, g = h.float() * rstd[:, None], dy.float() * gamma.float()
        dh = rstd[:, None] * (g - xh * (g * xh).mean(1, keepdim=True)) + (0 if dres is None else dres.float())
        return dh.to(h.dtype), (dy.float() * xh).sum(0) if need_dgamma else None

    def te_cast_fp8_per_token_transpose(self, x, dtype, flags=0):
        self.said("cast")
        return x.float(), None, x.float().t().contiguous(), None

    def te_fp8_gemm_fwd(self, a, sa, da, b, sb, db, bias=None, epilogue=0, preact=None, y_dtype=None, accum=0):
        self.said("fwd")
        z = a @ b.t() + (0 if bias is None else bias.float())
        if preact is not None:
            preact.copy_(z)
        return (torch.nn.functional.gelu(z, approximate="tanh") if epilogue & te.TE_EPI_GELU else z).bfloat16()

    def te_fp8_gemm_dgrad(self, a, sa, da, b, sb, db, epilogue=0, preact=None, dx_dtype=None, accum=0):
        self.said("dgrad")
        return self._dgrad(a, b, preact).bfloat16()

    def te_fp8_gemm_dgrad_deterministic(self, a, sa, da, b, sb, db, bias_grad, epilogue=0, preact=None, dx_dtype=None, accum=0):
        self.said("dgrad")
        d = self._dgrad(a, b, preact)
        bias_grad.copy_(d.sum(0))
        return d.bfloat16()

    def _dgrad(self, a, b, preact):
        d = a @ b.t()
        if preact is not None:
            with torch.enable_grad():
                z = preact.float().requires_grad_()
                torch.nn.functional.gelu(z, approximate="tanh").sum().backward()
            d = d * z.grad
        return d

    def te_fp8_wgrad_accum(self, a, sa, da, b, sb, db, out, accum):
        self.said("wgrad")
        out += a @ b.t()

    def te_fp8_wgrad_accum_bgrad(self, a, sa, da, b, sb, db, out, bias_grad, accum):
        self.said("wgrad")
        out += a @ b.t()
        bias_grad.copy_(a.sum(1))

    def te_moe_router_fwd(self, logits, top_k, renormalize=False, token_mask=None, loss=False, need_lse=None):
        p = torch.softmax(logits.float(), 1)
        w, index = p.topk(top_k, 1)
        counts = torch.bincount(index.reshape(-1), minlength=p.shape[1]).int()
        return RouterOutput(index.int(), w, torch.logsumexp(logits.float(), 1), counts, torch.tensor([len(p)], dtype=torch.int32),
                            (counts * p.sum(0)).sum().reshape(1) * p.shape[1] / (top_k * len(p) ** 2))

    def te_moe_router_bwd(self, logits, index, lse, counts=None, routed=None, d_weight=None, d_loss=None, renormalize=False):
        p = torch.exp(logits.float() - lse[:, None])
        b = torch.zeros_like(p)
        if d_loss is not None:
            b += d_loss * p.shape[1] / index.shape[1] * counts.float() / len(p) ** 2
        if d_weight is not None:
            b.scatter_add_(1, index.long(), d_weight)
        return (p * (b - (p * b).sum(1, keepdim=True))).to(logits.dtype)

    def te_grad_norm_clip(self, grads, max_norm):
        self.said("clip", count=len(grads))
        norm = torch.sqrt(sum((g.double() ** 2).sum() for g in grads)).float().reshape(1)
        for g in grads:
            g.mul_(min(1.0, max_norm / (float(norm) + 1e-6)))
        return norm


@pytest.fixture
def calls(monkeypatch):
    c = Calls()
    for module in (block, linear):
        for name in dir(c):
            if name.startswith("te_") and hasattr(module, name):
                monkeypatch.setattr(module, name, getattr(c, name))
    return c


def randn(shape, seed, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype)


def close(a, b):
    """Within eight half steps of bf16 of the largest value (the intermediate results are stored in bf16)."""
    return bool(((a.double() - b.double()).abs() <= 8 * 2.0 ** -8 * b.double().abs().max()).all())


def norm_mlp(main_grad=True):
    m = block.Fp8NormMlp(128, 256, 128, device="cpu", generator=torch.Generator().manual_seed(0))
    m.mlp.b1.data.copy_(randn((256,), 5, 0.1))
    m.mlp.b2.data.copy_(randn((128,), 6, 0.1))
    if not main_grad:
        for p in (m.norm.weight, m.mlp.w1, m.mlp.w2):
            del p.main_grad
    return m


PARAMS = ("norm.weight", "mlp.w1", "mlp.b1", "mlp.w2", "mlp.b2")


def got(p):
    main = getattr(p, "main_grad", None)
    return main if main is not None else p.grad


def reference(m, x, res, dy, dh):
    """Gradients by autograd of the block in fp32: x, residual and the parameters."""
    leaves = [t.detach().float().requires_grad_() for t in (x, res, *(m.get_parameter(n) for n in PARAMS))]
    x32, r32, g, w1, b1, w2, b2 = leaves
    h = x32 + r32
    n = h * torch.rsqrt((h * h).mean(1, keepdim=True) + 1e-5) * g
    y = torch.nn.functional.gelu(n @ w1.t() + b1, approximate="tanh") @ w2.t() + b2
    torch.autograd.backward([y, h], [dy.float(), dh.float()])
    return [t.grad for t in leaves]


# ------------------------------------------------------------------ frozen parameters
@pytest.mark.parametrize("main_grad", [False, True])
def test_a_frozen_norm_weight_gets_no_gradient(calls, main_grad):
    m = block.RmsNorm(64, device="cpu", main_grad=main_grad)
    m.weight.requires_grad_(False)
    x = randn((6, 64), 1).requires_grad_()
    y, _ = m(x)
    y.backward(randn(y.shape, 2))
    assert x.grad is not None and m.weight.grad is None
    assert not main_grad or bool((m.weight.main_grad == 0).all())
    assert [o["need_dgamma"] for o in calls.options if o["name"] == "norm_bwd"] == [False]


@pytest.mark.parametrize("main_grad", [False, True])
@pytest.mark.parametrize("frozen", [(), ("norm.weight",), ("mlp.w1",), ("mlp.w2",), ("mlp.w1", "mlp.w2"), ("mlp.b1", "mlp.b2"),
                                    ("mlp.w1", "mlp.b1"), ("mlp.w2", "mlp.b2"), PARAMS, PARAMS[:4], PARAMS[1:], PARAMS[:1] + PARAMS[2:]],
                         ids="+".join)
@pytest.mark.parametrize("inputs", [True, False])
def test_norm_mlp_with_frozen_parameters(calls, frozen, inputs, main_grad):
    """Every gradient that is asked for, and nothing added to what is frozen."""
    if not inputs and set(frozen) == set(PARAMS):
        pytest.skip("nothing takes a gradient")
    m = norm_mlp(main_grad)
    for n in frozen:
        m.get_parameter(n).requires_grad_(False)
    x, res = randn((128, 128), 1).requires_grad_(inputs), randn((128, 128), 2).requires_grad_(inputs)
    y, h = m(x, res)
    dy, dh = randn(y.shape, 3, 0.1), randn(h.shape, 4, 0.1)
    want = reference(m, x, res, dy, dh)
    del calls.log[:], calls.options[:]
    torch.autograd.backward([y, h], [dy, dh]) if h.requires_grad else y.backward(dy)
    if inputs:
        assert close(x.grad, want[0]) and close(res.grad, want[1])
    for n, w in zip(PARAMS, want[2:]):
        p = m.get_parameter(n)
        if n in frozen:
            assert p.grad is None and bool((getattr(p, "main_grad", torch.zeros(1)) == 0).all()), n
        else:
            assert close(got(p), w), n
    assert [o["need_dgamma"] for o in calls.options if o["name"] == "norm_bwd"] in ([], ["norm.weight" not in frozen])
    # products of the weights' gradients: of those that are asked for (fc2's brings its bias gradient)
    assert calls.log.count("wgrad") == ("mlp.w1" not in frozen) + (not {"mlp.w2", "mlp.b2"} <= set(frozen))


def test_a_frozen_fc1_needs_no_transposed_operand(calls):
    m = norm_mlp()
    x = randn((128, 128), 1).requires_grad_()
    m(x)
    m.mlp.w1.requires_grad_(False)
    m(x)
    assert [o["transpose"] for o in calls.options if o["name"] == "norm"] == [True, False]


# ------------------------------------------------------------------ clip_grad_norm
def test_clip_leaves_frozen_parameters_out(calls):
    """A frozen parameter's buffer (here one filled before it was frozen) neither counts nor changes."""
    a, b, c = (torch.nn.Parameter(torch.zeros(4, dtype=torch.bfloat16)) for _ in range(3))
    a.main_grad, b.main_grad = torch.full((4,), 3.0), torch.full((4,), 100.0)
    b.requires_grad_(False)
    c.grad = torch.full((4,), 100.0, dtype=torch.bfloat16)
    c.requires_grad_(False)
    norm = block.clip_grad_norm([a, b, c], 3.0)
    assert float(norm) == 6.0
    assert torch.allclose(a.main_grad, torch.full((4,), 1.5)) and bool((b.main_grad == 100).all()) and bool((c.grad == 100).all())


def test_clip_takes_a_shared_parameter_once(calls):
    """A weight that two modules share comes twice in their parameters: clipped twice, its two passes would race."""
    a, b = (torch.nn.Parameter(torch.zeros(4, dtype=torch.bfloat16)) for _ in range(2))
    a.main_grad, b.main_grad = torch.full((4,), 3.0), torch.full((4,), 4.0)
    norm = block.clip_grad_norm([a, b, a], 5.0)
    assert float(norm) == 10.0 and calls.options[-1]["count"] == 2
    assert torch.allclose(a.main_grad, torch.full((4,), 1.5)) and torch.allclose(b.main_grad, torch.full((4,), 2.0))


def test_clip_takes_one_parameter_for_a_list(calls):
    """As torch's function does; its rows, taken for parameters, have no gradients, and nothing was clipped."""
    a = torch.nn.Parameter(torch.zeros(4, 4, dtype=torch.bfloat16))
    a.main_grad = torch.full((4, 4), 2.0)
    assert float(block.clip_grad_norm(a, 4.0)) == 8.0 and torch.allclose(a.main_grad, torch.ones(4, 4))


# ------------------------------------------------------------------ linear.py
@pytest.mark.parametrize("main_grad", [False, True])
@pytest.mark.parametrize("train", ["x", "w", "b", "xw", "xb", "wb", "xwb"])
def test_linear_with_frozen_parameters(calls, train, main_grad):
    m = linear.Fp8Linear(128, 256, device="cpu", generator=torch.Generator().manual_seed(0), fuse_wgrad_accumulation=main_grad)
    m.weight.requires_grad_("w" in train)
    m.bias.requires_grad_("b" in train)
    x = randn((128, 128), 1).requires_grad_("x" in train)
    y = m(x)
    dy = randn(y.shape, 2, 0.1)
    y.backward(dy)
    assert ("x" in train) == (x.grad is not None)
    if "x" in train:
        assert close(x.grad, dy.float() @ m.weight.detach().float())
    if "w" in train:
        assert close(got(m.weight), dy.float().t() @ x.detach().float())
    else:
        assert m.weight.grad is None and bool((getattr(m.weight, "main_grad", torch.zeros(1)) == 0).all())
    assert close(m.bias.grad, dy.float().sum(0)) if "b" in train else m.bias.grad is None
    assert calls.log.count("wgrad") == ("w" in train or "b" in train) and calls.log.count("dgrad") == ("x" in train)


@pytest.mark.parametrize("main_grad", [False, True])
@pytest.mark.parametrize("frozen", [(), ("w1",), ("w2",), ("w1", "w2"), ("b1", "b2"), ("w1", "b1"), ("w2", "b2"),
                                    ("w1", "b1", "w2", "b2"), ("w1", "b1", "b2"), ("b1", "w2", "b2")], ids="+".join)
@pytest.mark.parametrize("inputs", [True, False])
def test_mlp_with_frozen_parameters(calls, frozen, inputs, main_grad):
    names = ("w1", "b1", "w2", "b2")
    if not inputs and set(frozen) == set(names):
        pytest.skip("nothing takes a gradient")
    m = linear.Fp8Mlp(128, 256, 128, device="cpu", generator=torch.Generator().manual_seed(0), fuse_wgrad_accumulation=main_grad)
    m.b1.data.copy_(randn((256,), 5, 0.1))
    for n in frozen:
        m.get_parameter(n).requires_grad_(False)
    x = randn((128, 128), 1).requires_grad_(inputs)
    y = m(x)
    dy = randn(y.shape, 3, 0.1)
    leaves = [t.detach().float().requires_grad_() for t in (x, m.w1, m.b1, m.w2, m.b2)]
    x32, w1, b1, w2, b2 = leaves
    (torch.nn.functional.gelu(x32 @ w1.t() + b1, approximate="tanh") @ w2.t() + b2).backward(dy.float())
    del calls.log[:]
    y.backward(dy)
    assert not inputs or close(x.grad, x32.grad)
    for n, w in zip(names, leaves[1:]):
        p = m.get_parameter(n)
        if n in frozen:
            assert p.grad is None and bool((getattr(p, "main_grad", torch.zeros(1)) == 0).all()), n
        else:
            assert close(got(p), w.grad), n
    assert calls.log.count("wgrad") == ("w1" not in frozen) + (not {"w2", "b2"} <= set(frozen))


# ------------------------------------------------------------------ second derivatives
def first_gradients(make, inputs, params):
    """The module's outputs that take a gradient, and their gradients with the graph kept."""
    outs = [o for o in make(*inputs) if o is not None and o.requires_grad and o.is_floating_point() and o.numel()]
    leaves = [t for t in (*inputs, *params) if t is not None and t.requires_grad]
    value = sum((o.float() * randn(o.shape, 9 + i, dtype=torch.float32)).sum() for i, o in enumerate(outs))
    return leaves, torch.autograd.grad(value, leaves, create_graph=True, allow_unused=True)


def second_order_cases():
    def norm(residual, train=True):
        m = block.RmsNorm(64, device="cpu", main_grad=False)
        m.weight.requires_grad_(train)
        res = randn((6, 64), 2).requires_grad_() if residual else None
        return m, (randn((6, 64), 1).requires_grad_(), res), (m.weight,)

    def mlp(cls, frozen=()):
        m = cls(128, 256, 128, device="cpu", generator=torch.Generator().manual_seed(0))
        for n, p in m.named_parameters():
            p.requires_grad_(n not in frozen)
            if hasattr(p, "main_grad"):
                del p.main_grad
        run = m if cls is block.Fp8NormMlp else lambda x: (m(x),)
        return run, (randn((128, 128), 1).requires_grad_(),), tuple(m.parameters())

    def linear_(train):
        m = linear.Fp8Linear(128, 256, device="cpu", generator=torch.Generator().manual_seed(0), fuse_wgrad_accumulation=False)
        m.weight.requires_grad_(train)
        return lambda x: (m(x),), (randn((128, 128), 1).requires_grad_(),), (m.weight, m.bias)

    def router(renormalize):
        m = block.TopKRouter(2, renormalize)
        return lambda v: m(v)[:2], (randn((6, 8), 1, dtype=torch.float32).requires_grad_(),), ()

    mlp_names, weights = ("w1", "b1", "w2", "b2"), ("norm.weight", "mlp.w1", "mlp.w2")
    return dict(norm=lambda: norm(False), norm_residual=lambda: norm(True), norm_frozen=lambda: norm(False, False),
                norm_mlp=lambda: mlp(block.Fp8NormMlp), norm_mlp_frozen=lambda: mlp(block.Fp8NormMlp, weights),
                mlp=lambda: mlp(linear.Fp8Mlp), mlp_frozen=lambda: mlp(linear.Fp8Mlp, mlp_names),
                linear=lambda: linear_(True), linear_frozen=lambda: linear_(False), router=lambda: router(False))


@pytest.mark.parametrize("case", list(second_order_cases()))
def test_second_derivatives_are_refused(calls, case):
    """Any value made of the first gradients: differentiated for the inputs, or for any parameter, it raises; the
    first gradients themselves are those without create_graph."""
    make, inputs, params = second_order_cases()[case]()
    leaves, first = first_gradients(make, inputs, params)
    plain = torch.autograd.grad(sum((o.float() * randn(o.shape, 9 + i, dtype=torch.float32)).sum() for i, o in enumerate(
        [o for o in make(*inputs) if o is not None and o.requires_grad and o.is_floating_point() and o.numel()])), leaves, allow_unused=True)
    assert all((a is None) == (b is None) and (a is None or torch.equal(a, b)) for a, b in zip(first, plain))
    for g in first:
        penalty = g.float().square().sum()
        for leaf in leaves:
            with pytest.raises(RuntimeError, match="second derivative"):
                torch.autograd.grad(penalty, [leaf], retain_graph=True, allow_unused=True)
        with pytest.raises(RuntimeError, match="second derivative"):
            (penalty + sum(t.float().sum() for t in leaves)).backward(retain_graph=True)


def test_first_derivatives_beside_a_second_one_elsewhere(calls):
    """create_graph=True for the sake of another part of the model: the modules' own gradients stay usable."""
    m = block.RmsNorm(64, device="cpu", main_grad=False)
    x = randn((6, 64), 1, dtype=torch.float32).requires_grad_()
    a = randn((64,), 2, dtype=torch.float32).requires_grad_()
    y, _ = m(x)
    value = (y.float() * 2).sum() + (a ** 3).sum()
    gx, ga = torch.autograd.grad(value, [x, a], create_graph=True)
    assert torch.equal(torch.autograd.grad(ga.sum(), a)[0], 6 * a.detach()) and bool((gx != 0).any())


@pytest.mark.parametrize("cls", ["norm", "mlp"])
def test_the_sum_alone_can_be_differentiated_again(calls, cls):
    """h = x + residual is an addition: where only it is used, its gradient is handed on with its graph."""
    m = norm_mlp() if cls == "mlp" else block.RmsNorm(128, device="cpu")
    x, res = (randn((128, 128), i, dtype=torch.float32).requires_grad_() for i in (1, 2))
    _, h = m(x, res)
    g, = torch.autograd.grad((h ** 3).sum(), x, create_graph=True)
    again, = torch.autograd.grad(g.sum(), res)
    assert torch.allclose(again, 6 * h.detach())
