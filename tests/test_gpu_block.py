"""The modules on the operators (block.py) and the example that runs them together.

The norm's output bound is u = 2^-24 work against a stored bf16 (half a step, 2^-8); whole modules are
compared with torch in fp32 on the same weights where no fp8 is between, and call by call where there is."""
import importlib.util
import os

import pytest
import torch

te = pytest.importorskip("fp8_linear_layer_amd")
pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    te.load_library()
    global block
    from fp8_linear_layer_amd import block


def randn(shape, seed, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def norm64(h, w, eps):
    h = h.double()
    return h * torch.rsqrt((h * h).mean(-1, keepdim=True) + eps) * w.double()


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("main_grad", [False, True])
def test_rms_norm_module(residual, main_grad):
    """y and the gradients against autograd through the formula in 64 bits (on the stored sum)."""
    m = block.RmsNorm(320, main_grad=main_grad)
    m.weight.data.copy_(randn((320,), 1, 0.1) + 1)
    x = randn((4, 33, 320), 2).requires_grad_()
    res = randn((4, 33, 320), 3, 2.0).requires_grad_() if residual else None
    y, h = m(x, res)
    dy, dh = randn(y.shape, 4), randn(y.shape, 5)
    torch.autograd.backward([y, h], [dy, dh]) if residual else y.backward(dy)

    h64 = h.detach().double().requires_grad_()
    w64 = m.weight.detach().double().requires_grad_()
    y64 = norm64(h64, w64, m.eps)
    ((y64 * dy.double()).sum() + ((h64 * dh.double()).sum() if residual else 0.0)).backward()
    assert ((y.double() - y64).abs() <= y64.abs() * (2.0 ** -8 + 40 * 2.0 ** -24)).all()
    # 80 u of the terms (|dy w| and the row's mean of them times |h| / rms, both times 1 / rms), and the bf16 store
    r = torch.rsqrt((h64.detach() ** 2).mean(-1, keepdim=True) + m.eps)
    g = (dy.double() * w64.detach()).abs()
    mag = r * (g + h64.detach().abs() * r * (g * h64.detach().abs() * r).mean(-1, keepdim=True)) + (dh.double().abs() if residual else 0)
    tol = 80 * 2.0 ** -24 * mag + h64.grad.abs() * 2.0 ** -8
    assert ((x.grad.double() - h64.grad).abs() <= tol).all()
    if residual:
        assert torch.equal(res.grad, x.grad)
    got = m.weight.main_grad if main_grad else m.weight.grad
    assert (m.weight.grad is None) == main_grad
    mag = (dy.double() * h64.detach() * r).abs().sum((0, 1))
    assert ((got.double() - w64.grad).abs() <= 80 * 2.0 ** -24 * mag + (0 if main_grad else w64.grad.abs() * 2.0 ** -8)).all()


@pytest.mark.parametrize("pow2", [False, True])
def test_norm_mlp_is_norm_and_mlp(pow2):
    """Fp8NormMlp gives what the library's own calls give one by one, bit for bit."""
    T, K, H = 256, 384, 512
    gen = torch.Generator(device="cuda").manual_seed(0)
    m = block.Fp8NormMlp(K, H, generator=gen, pow2_scales=pow2)
    m.norm.weight.data.copy_(randn((K,), 1, 0.1) + 1)
    x, res = randn((T, K), 2).requires_grad_(), randn((T, K), 3, 2.0).requires_grad_()
    y, h = m(x, res)
    dy, dh = randn(y.shape, 4, 1e-3), randn(h.shape, 5, 1e-3)
    torch.autograd.backward([y, h], [dy, dh])

    flags, accum = (te.TE_CAST_POW2_SCALE, te.TE_ACCUM_FAST) if pow2 else (0, te.TE_ACCUM_FULL_FP32)
    E4, E5 = te.TE_DTYPE_E4M3, te.TE_DTYPE_E5M2
    n = te.te_rmsnorm_fwd(x.detach(), m.norm.weight.detach(), m.norm.eps, residual=res.detach(), out_dtype=E4, flags=flags, transpose=True)
    assert torch.equal(h, n.h)
    w1, w2 = m.mlp.w1.detach(), m.mlp.w2.detach()
    qw1, sw1, qw1t, sw1t = te.te_cast_fp8_per_token_transpose(w1, E4, flags)
    qw2, sw2, qw2t, sw2t = te.te_cast_fp8_per_token_transpose(w2, E4, flags)
    z = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    a = te.te_fp8_gemm_fwd(n.q, n.scales, E4, qw1, sw1, E4, bias=m.mlp.b1.detach(), preact=z, accum=accum,
                           epilogue=te.TE_EPI_BIAS | te.TE_EPI_GELU | te.TE_EPI_AUX_PREACT)
    qa, sa, qat, sat = te.te_cast_fp8_per_token_transpose(a, E4, flags)
    assert torch.equal(y, te.te_fp8_gemm_fwd(qa, sa, E4, qw2, sw2, E4, bias=m.mlp.b2.detach(), epilogue=te.TE_EPI_BIAS, accum=accum))
    qd, sd, _, _ = te.te_cast_fp8_per_token_transpose(dy, E5)
    db = torch.empty((H,), dtype=torch.float32, device="cuda")
    dz = te.te_fp8_gemm_dgrad_deterministic(qd, sd, E5, qw2t, sw2t, E4, db, epilogue=te.TE_EPI_DGELU | te.TE_EPI_BGRAD, preact=z)
    qz, sz, qzt, szt = te.te_cast_fp8_per_token_transpose(dz, E5)
    dn = te.te_fp8_gemm_dgrad(qz, sz, E5, qw1t, sw1t, E4)
    want, dgamma = te.te_rmsnorm_bwd(dn, n.h, n.rstd, m.norm.weight.detach(), dres=dh)
    assert torch.equal(x.grad, want) and torch.equal(res.grad, want) and torch.equal(m.norm.weight.main_grad, dgamma)
    dw1 = torch.zeros((H, K), dtype=torch.float32, device="cuda")
    te.te_fp8_wgrad_accum(qzt, szt, E5, n.qt, n.scales_t, E4, dw1)
    assert torch.equal(m.mlp.w1.main_grad, dw1)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("use", ["both", "weight", "loss"])
def test_router_module(renorm, use):
    """Gradients of the logits against autograd through the formula in 64 bits."""
    tokens, experts, k = 300, 24, 3
    logits = randn((tokens, experts), 1, dtype=torch.float32).requires_grad_()
    mask = torch.arange(tokens, device="cuda") % 5 != 0
    weight, loss, index, counts = block.TopKRouter(k, renorm)(logits, mask)
    assert not index.requires_grad and not counts.requires_grad
    dw = randn(weight.shape, 2, dtype=torch.float32)
    value = (weight * dw).sum() * (use != "loss") + loss[0] * (use != "weight")
    value.backward()
    v = logits.detach().double().requires_grad_()
    p = torch.softmax(v, 1)
    ok = index >= 0
    w = torch.where(ok, p.gather(1, index.long().clamp_min(0)), 0.0)
    if renorm:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    n = int(mask.sum())
    l64 = experts / k * (counts.double() * (p * mask[:, None]).sum(0)).sum() / n ** 2
    ((w * dw.double()).sum() * (use != "loss") + l64 * (use != "weight")).backward()
    # 160 u of the terms: each is p (or w) times at most twice the largest |d_weight| or coefficient of the loss
    top = p.detach() * 2 * (dw.abs().double().sum(1, keepdim=True) * (use != "loss") + experts / k * counts.max() / n ** 2)
    if renorm:
        top = top.scatter_add(1, index.long().clamp_min(0), 2 * w.detach() * dw.abs().double().sum(1, keepdim=True))
    assert ((logits.grad.double() - v.grad).abs() <= 160 * 2.0 ** -24 * top).all()


def test_clip_grad_norm_takes_main_grad():
    a, b, c = (torch.nn.Parameter(torch.zeros(5, dtype=torch.bfloat16, device="cuda")) for _ in range(3))
    a.main_grad = torch.full((5,), 3.0, device="cuda")
    b.grad = torch.full((5,), 4.0, dtype=torch.bfloat16, device="cuda")
    norm = block.clip_grad_norm([a, b, c], 1.0)
    assert abs(float(norm) - 125 ** 0.5) <= 2.0 ** -23 * 125 ** 0.5
    assert torch.allclose(a.main_grad, torch.full((5,), 3 / 125 ** 0.5, device="cuda")) and c.grad is None
    assert float(b.grad[0]) == float(torch.tensor(4 / 125 ** 0.5).bfloat16())


def test_example_learns():
    spec = importlib.util.spec_from_file_location("moe_block_step", os.path.join(ROOT, "examples", "moe_block_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    history = m.main(["--tokens", "512", "--width", "256", "--hidden", "384", "--experts", "5", "--steps", "8"])
    losses = [h[0] for h in history]
    assert losses[-1] < 0.8 * losses[0], losses
    assert all(h[2] == h[2] and h[2] > 0 and 0.9 <= h[1] < 5 for h in history)
