"""GPU parity of te_grad_norm_clip with the formula in 64 bits.

The sums are in 64 bits, so the norm is off by its one rounding to fp32 (2^-24; twice that is allowed); the
coefficient and the product add four roundings, and the store half a step of the output's type."""
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


def tensors(sizes, dtype, seed, std=1e-3):
    g = gen(seed)
    return [(torch.randn(n, generator=g, device="cuda") * std).to(dtype) for n in sizes]


def exact(grads, max_norm):
    total = sum(float(g.double().square().sum()) for g in grads)
    norm = total ** 0.5
    return norm, min(1.0, max_norm / (norm + 1e-6))


def check(grads, max_norm, norm, outs):
    want, coef = exact(grads, max_norm)
    assert abs(float(norm) - want) <= 2 * U * want
    for g, o in zip(grads, outs):
        w = g.double() * coef
        assert ((o.double() - w).abs() <= (HALF[o.dtype] + 6 * U) * w.abs() + 2.0 ** -133).all()


SIZES = [[1], [7], [8], [8191], [8192], [8193], [100003], [3, 0, 20000, 1, 9], [0], [0, 0, 5], [17] * 40, [33] * 96, [33] * 97, [129] * 300]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("gt,ot", [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32"), ("bf16", "bf16")])
def test_clip(sizes, gt, ot):
    for max_norm in (1e-4, 1e6):
        grads = tensors(sizes, DT[gt], len(sizes))
        outs = [torch.full_like(g, 7.0, dtype=DT[ot]) for g in grads]
        norm = te.te_grad_norm_clip(grads, max_norm, out=outs)
        check(grads, max_norm, norm, outs)
        again = te.te_grad_norm_clip(grads, max_norm, out=outs)
        assert torch.equal(norm, again)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_in_place(dtype):
    for max_norm in (1e-4, 1e6):
        grads = tensors([5, 9000, 64], DT[dtype], 3)
        before = [g.clone() for g in grads]
        norm = te.te_grad_norm_clip(grads, max_norm)
        check(before, max_norm, norm, grads)
        if max_norm == 1e6:
            assert all(torch.equal(a, b) for a, b in zip(before, grads))


def test_types_mixed_and_neighbours_in_one_buffer():
    """Gradients cut from buckets at odd offsets; the elements around them stay."""
    sizes = [3, 8190, 1, 10000, 77]
    f, b = torch.randn(20000, generator=gen(1), device="cuda"), torch.randn(20000, generator=gen(2), device="cuda").bfloat16()
    of, ob = torch.full((20000,), 7.0, device="cuda"), torch.full((20000,), 7.0, device="cuda").bfloat16()
    grads, outs, at = [], [], 1
    for i, n in enumerate(sizes):
        grads.append((f, b)[i % 2][at:at + n])
        outs.append((of, ob)[(i // 2) % 2][at:at + n])
        at += n + 1
    norm = te.te_grad_norm_clip(grads, 0.5, out=outs)
    check(grads, 0.5, norm, outs)
    for buf in (of, ob):
        keep = torch.ones(20000, dtype=torch.bool, device="cuda")
        for o in outs:
            if o.untyped_storage().data_ptr() == buf.data_ptr():
                keep[o.storage_offset():o.storage_offset() + o.numel()] = False
        assert (buf[keep] == 7.0).all()


def test_dense_tensors_of_another_order():
    g = torch.randn((40, 50), generator=gen(1), device="cuda").t()
    o = torch.empty((40, 50), device="cuda").t()
    norm = te.te_grad_norm_clip([g], 1.0, out=[o])
    check([g], 1.0, norm, [o])
    with pytest.raises(te.TeFp8Error, match="layout"):
        te.te_grad_norm_clip([g], 1.0, out=[torch.empty((50, 40), device="cuda")])
    with pytest.raises(te.TeFp8Error, match="layout"):
        te.te_grad_norm_clip([torch.zeros((8, 8), device="cuda")[:, ::2]], 1.0)


def test_values_whose_squares_leave_fp32():
    for scale in (1e30, 1e-35):
        grads = tensors([1000, 31], torch.float32, 4, std=scale)
        outs = [torch.empty_like(g) for g in grads]
        norm = te.te_grad_norm_clip(grads, 1.0, out=outs)
        want, coef = exact(grads, 1.0)
        assert abs(float(norm) - want) <= 2 * U * want + 2.0 ** -149
        if scale > 1:
            check(grads, 1.0, norm, outs)


def test_nan_and_infinity():
    grads = tensors([100, 50], torch.float32, 5)
    grads[1][3] = INF
    outs = [torch.empty_like(g) for g in grads]
    norm = te.te_grad_norm_clip(grads, 1.0, out=outs)
    assert float(norm) == INF and (outs[0] == 0).all() and outs[1][3].isnan() and (outs[1][4:] == 0).all()
    grads[0][0] = NAN
    norm = te.te_grad_norm_clip(grads, 1.0, out=outs)
    assert norm.isnan() and all(o.isnan().all() for o in outs)


def test_no_gradients():
    norm = te.te_grad_norm_clip([], 1.0)
    assert float(norm) == 0.0


def test_more_elements_than_31_bits():
    n = (1 << 31) + 12345
    g = torch.zeros((n,), dtype=torch.bfloat16, device="cuda")
    g[0], g[n - 1], g[1 << 31] = 3.0, 4.0, 12.0
    out = torch.empty_like(g)
    norm = te.te_grad_norm_clip([g], 6.5, out=[out])
    assert float(norm) == 13.0
    assert float(out[0]) == 1.5 and float(out[n - 1]) == 2.0 and float(out[1 << 31]) == 6.0 and int((out != 0).sum()) == 3


@pytest.mark.parametrize("gt", ["f32", "bf16"])
@pytest.mark.parametrize("ot", ["f32", "bf16"])
def test_totals_larger_than_the_caches(gt, ot):
    """16384 chunks and more go past the caches; tensors at odd offsets and of odd sizes."""
    sizes = [100_000_003, 5, 35_000_001]
    g = gen(8)
    flat = (torch.randn(sum(sizes) + 1, generator=g, device="cuda") * 1e-3).to(DT[gt])
    out = torch.full((sum(sizes) + 3,), 7.0, dtype=DT[ot], device="cuda")
    grads, outs = list(flat[1:].split(sizes)), list(out[1:-2].split(sizes))
    norm = te.te_grad_norm_clip(grads, 1.0, out=outs)
    check(grads, 1.0, norm, outs)
    assert out[0] == 7.0 and (out[-2:] == 7.0).all()


def test_given_stream():
    grads = tensors([50000, 3], torch.float32, 7)
    outs = [torch.empty_like(g) for g in grads]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    norm = te.te_grad_norm_clip(grads, 1e-3, out=outs, stream=side)
    side.synchronize()
    check(grads, 1e-3, norm, outs)


def test_other_stream_and_graph():
    grads = tensors([5000, 77, 20001], torch.float32, 6)
    outs = [torch.empty_like(g, dtype=torch.bfloat16) for g in grads]

    def step():
        norm = te.te_grad_norm_clip(grads, 1e-3, out=outs)
        return [norm] + [o.clone() for o in outs]

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
        for g in grads:
            g.normal_(generator=gen(60 + i))
        graph.replay()
        torch.cuda.synchronize()
        replayed = [o.clone() for o in out]
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(replayed, eager)), i
