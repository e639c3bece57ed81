"""te_grad_norm_clip over more tensors than one launch takes: the partial sums of all launches are right however
many workgroups each has, and repeat.  Tolerances as for few tensors: the norm in 64-bit sums, one rounding to fp32."""
import pytest
import torch

te = pytest.importorskip("fp8_linear_layer_amd")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
SMALL, LARGE, HUGE = 5, 40000, 9_000_000
LISTS = {
    "small then large": [SMALL] * 96 + [LARGE] * 200,
    "large then small": [LARGE] * 200 + [SMALL] * 300,
    "small, all workgroups, small": [SMALL] * 96 + [HUGE] + [SMALL] * 300,
    "empty ones between": ([0, SMALL, 0, LARGE] * 150),
    "a launch of empty ones": [SMALL] * 96 + [0] * 500 + [LARGE] * 97,
    "2000": [(37 * i) % 3000 + 1 for i in range(2000)],
}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    te.load_library()


def make(sizes, dtype, seed):
    flat = (torch.randn(sum(sizes), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda") * 1e-3).to(dtype)
    return flat, list(flat.split(sizes))


@pytest.mark.parametrize("name", list(LISTS))
@pytest.mark.parametrize("gt,ot", [(torch.float32, torch.float32), (torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)])
def test_norm_and_outputs(name, gt, ot):
    sizes = LISTS[name]
    flat, grads = make(sizes, gt, 1)
    out = torch.full((sum(sizes),), 7.0, dtype=ot, device="cuda")
    workspace = torch.full((te.ops._lib().te_grad_norm_workspace_bytes(len(sizes)),), 0xFF, dtype=torch.uint8, device="cuda")   # NaN
    norm = te.te_grad_norm_clip(grads, 0.01, out=list(out.split(sizes)), workspace=workspace)
    want = float(flat.double().square().sum().sqrt())
    assert abs(float(norm) - want) <= 2 * U * want
    w = flat.double() * min(1.0, 0.01 / (want + 1e-6))
    assert ((out.double() - w).abs() <= (HALF[ot] + 6 * U) * w.abs() + 2.0 ** -133).all()
    first = out.clone()
    again = te.te_grad_norm_clip(grads, 0.01, out=list(out.split(sizes)), workspace=workspace)
    assert torch.equal(norm, again) and torch.equal(first, out)


@pytest.mark.parametrize("at", [0, 200, 499])
def test_nan_in_any_launch(at):
    flat, grads = make([100] * 500, torch.float32, 2)
    grads[at][3] = float("nan")
    norm = te.te_grad_norm_clip(grads, 1.0)
    assert norm.isnan() and flat.isnan().all()


def test_graph():
    """Replays with new gradients and eager calls between them."""
    sizes = LISTS["small then large"]
    flat, grads = make(sizes, torch.float32, 3)
    out = torch.empty_like(flat)
    outs = list(out.split(sizes))
    te.te_grad_norm_clip(grads, 0.01, out=outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = te.te_grad_norm_clip(grads, 0.01, out=outs)
    for i in range(4):
        flat.normal_(generator=torch.Generator(device="cuda").manual_seed(10 + i))
        graph.replay()
        torch.cuda.synchronize()
        got, replayed = out.clone(), norm.clone()
        eager = te.te_grad_norm_clip(grads, 0.01, out=outs)
        torch.cuda.synchronize()
        assert torch.equal(eager, replayed) and torch.equal(out, got), i


@pytest.mark.parametrize("max_norm,touched", [(1.0, True), (1.0 + 2.0 ** -21, True), (1.0 + 2.0 ** -19, False), (2.0, False)])
def test_in_place_is_rewritten_where_the_coefficient_is_below_one(max_norm, touched):
    """A norm of 1 against limits at and just above it: 1e-6 is added to the norm before the division."""
    g = torch.zeros(9000, device="cuda")
    g[17] = 1.0
    norm = te.te_grad_norm_clip([g], max_norm)
    coef = torch.tensor(max_norm) / (torch.tensor(1.0) + torch.tensor(1e-6))
    assert float(norm) == 1.0 and float(g[17]) == min(1.0, float(coef)) and (float(g[17]) < 1.0) == touched
