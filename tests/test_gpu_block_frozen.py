"""Frozen parameters of the modules on the operators: their gradients are not computed and not accumulated, and
those of the others are, bit for bit, what they are when everything is trained."""
import pytest
import torch

te = pytest.importorskip("fp8_linear_layer_amd")
pytestmark = pytest.mark.gpu

PARAMS = ("norm.weight", "mlp.w1", "mlp.b1", "mlp.w2", "mlp.b2")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    te.load_library()
    global block
    from fp8_linear_layer_amd import block


def randn(shape, seed, std=1.0):
    return (torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda") * std).bfloat16()


def step(frozen):
    m = block.Fp8NormMlp(256, 384, 128, generator=torch.Generator(device="cuda").manual_seed(0))
    m.norm.weight.data.copy_(randn((256,), 1, 0.1) + 1)
    for n in frozen:
        m.get_parameter(n).requires_grad_(False)
    x, res = randn((256, 256), 2).requires_grad_(), randn((256, 256), 3, 2.0).requires_grad_()
    y, h = m(x, res)
    torch.autograd.backward([y, h], [randn(y.shape, 4, 1e-3), randn(h.shape, 5, 1e-3)])
    return m, x.grad, res.grad


@pytest.mark.parametrize("frozen", [("norm.weight",), ("mlp.w1", "mlp.w2"), ("mlp.w1", "mlp.b1"), ("mlp.w2", "mlp.b2"), PARAMS],
                         ids="+".join)
def test_norm_mlp(frozen):
    all_, gx, gr = step(())
    m, fx, fr = step(frozen)
    assert torch.equal(gx, fx) and torch.equal(gr, fr)
    for n in PARAMS:
        p, q = m.get_parameter(n), all_.get_parameter(n)
        if n in frozen:
            assert p.grad is None and bool((getattr(p, "main_grad", torch.zeros(1)) == 0).all()), n
        elif hasattr(p, "main_grad"):
            assert torch.equal(p.main_grad, q.main_grad) and bool((p.main_grad != 0).any()), n
        else:
            assert torch.equal(p.grad, q.grad), n


def test_norm():
    grads = []
    for train in (True, False):
        m = block.RmsNorm(2112)
        m.weight.requires_grad_(train)
        x = randn((77, 2112), 1).requires_grad_()
        y, _ = m(x)
        y.backward(randn(y.shape, 2))
        grads.append(x.grad)
        assert bool((m.weight.main_grad != 0).any()) == train
    assert torch.equal(*grads)


def test_create_graph():
    """First gradients with the graph kept are the plain ones, and differentiating them again raises."""
    m = block.RmsNorm(256, main_grad=False)
    x = randn((8, 256), 1).requires_grad_()
    dy = randn((8, 256), 2)
    plain = torch.autograd.grad(m(x)[0], [x, m.weight], dy)
    first = torch.autograd.grad(m(x)[0], [x, m.weight], dy, create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(plain, first))
    with pytest.raises(RuntimeError, match="second derivative"):
        first[0].float().square().sum().backward()
