"""Edges of te_layernorm_fwd / te_layernorm_bwd that test_gpu_layernorm leaves out: rows of less than eight columns far from
zero, fp8 outputs of one group, long rows of which a workgroup of the backward pass has several, and rates below fp32's
smallest.  Tolerances as there."""
import numpy as np
import pytest
import torch

import oracle
from parity import host, shost
from test_gpu_layernorm import DT, EPS, FMT, OUT, U, check_bwd, check_fwd, close, normal, rng, run_bwd, vector

te = pytest.importorskip("fp8_linear_layer_amd")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    te.load_library()


@pytest.mark.parametrize("cols", [1, 3, 5, 7])
@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("dres,p", [(False, 0.0), (True, 0.25)])
def test_backward_of_short_rows_far_from_zero(cols, t, dres, p):
    """A constant row of 2^126 has the deviation 0 and the finite gradient rstd (g - mean of g).  What stands behind a row's
    end is in none of its sums: 0 in h's place would give (0 - mean) rstd, which is infinite here."""
    rows = 37
    g = torch.Generator(device="cuda").manual_seed(cols)
    h = torch.full((rows, cols), 2.0 ** 126, dtype=DT[t], device="cuda")
    h[::2] *= -1
    mean, rstd = h[:, 0].float().contiguous(), torch.full((rows,), EPS ** -0.5, device="cuda")
    r = te.te_layernorm_fwd(h, vector(g, cols, 0.1, 1.0), None, EPS)
    assert torch.equal(r.mean, mean) and ((r.rstd - rstd).abs() <= 4 * U * rstd).all()
    dy, gamma = normal(g, (rows, cols), DT[t], 1e-2), vector(g, cols, 0.1, 1.0)
    res = normal(g, (rows, cols), DT[t], 1e-2) if dres else None
    got = te.te_layernorm_bwd(dy, h, mean, rstd, gamma, dres=res, p=p, rng=rng() if p else None)
    assert got.dh.isfinite().all()
    check_bwd((dy, h, mean, rstd, gamma, res), p, got)


@pytest.mark.parametrize("rows,cols", [(1, 128), (3, 128), (128, 128), (256, 64), (384, 8)])
@pytest.mark.parametrize("out", ["e4m3", "e5m2"])
@pytest.mark.parametrize("xt,ht,pow2,p", [("bf16", "bf16", False, 0.1), ("f32", "", True, 0.0), ("bf16", "f32", False, 0.0), ("f32", "bf16", True, 0.5)])
def test_fp8_outputs_of_one_group(rows, cols, out, xt, ht, pow2, p):
    g = torch.Generator(device="cuda").manual_seed(rows * 31 + cols)
    x = normal(g, (rows, cols), DT[xt], 0.7, 0.5)
    res = normal(g, (rows, cols), DT[ht], 2.0) if ht else None
    gamma, beta = vector(g, cols, 0.1, 1.0), vector(g, cols, 0.3)
    kw = dict(residual=res, p=p, rng=rng() if p else None)
    plain = te.te_layernorm_fwd(x, gamma, beta, EPS, out_dtype=te.TE_DTYPE_F32, **kw)
    y, bound = check_fwd(x, res, p, gamma, beta, plain)
    close(plain.y, y, bound + U * y.abs(), "y")
    assert (plain.y != 0).all(1).any()
    y32 = host(plain.y).numpy()
    for rowwise, transpose in ((True, False), (False, True), (True, True)):
        if (rowwise and cols % 128) or (transpose and rows % 128):
            continue
        r = te.te_layernorm_fwd(x, gamma, beta, EPS, out_dtype=OUT[out], flags=te.TE_CAST_POW2_SCALE if pow2 else 0, rowwise=rowwise,
                                transpose=transpose, **kw)
        for q, s, want, n in ((r.q, r.scales, y32, rows), (r.qt, r.scales_t, np.ascontiguousarray(y32.T), cols)):
            if q is None:
                continue
            oq, os_ = oracle.cast_per_token_f32(want, FMT[out], pow2)
            assert np.array_equal(host(q).numpy(), oq) and oq.any()
            assert np.array_equal(shost(s, n).view(np.uint32), os_.view(np.uint32))


@pytest.mark.parametrize("cols", [8200, 14336, 16384, 16392, 20003, 32768])
@pytest.mark.parametrize("yt,ht,dres,p", [("bf16", "bf16", True, 0.1), ("f32", "f32", False, 0.0), ("bf16", "f32", True, 0.3), ("f32", "bf16", True, 0.0)])
def test_backward_of_many_long_rows(cols, yt, ht, dres, p):
    """600 rows on a workgroup for each of 256 compute units: the loop over a workgroup's rows, with all outputs."""
    g = torch.Generator(device="cuda").manual_seed(cols)
    args, r = run_bwd(600, cols, yt, ht, dres, p, g, dx_dtype=OUT[yt])
    check_bwd(args, p, r)
    if args[5] is not None:     # and in place
        mine = args[5].clone()
        got = te.te_layernorm_bwd(*args[:5], dres=mine, p=p, rng=rng() if p else None, dh=mine, dx_dtype=OUT[yt])
        assert torch.equal(mine, r.dh) and torch.equal(got.dgamma, r.dgamma) and (not p or torch.equal(got.dx, r.dx))


@pytest.mark.parametrize("p", [1e-30, 1e-46, 1e-300])
def test_rates_too_small_for_fp32(p):
    """Such a rate drops nothing, as any below 2^-17, and the calls and the modules take it all the same."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x, res, dy = (normal(g, (9, 72), torch.bfloat16) for _ in range(3))
    gamma = vector(g, 72, 0.1, 1.0)
    want = te.te_layernorm_fwd(x, gamma, None, EPS, residual=res)
    r = te.te_layernorm_fwd(x, gamma, None, EPS, residual=res, p=p, rng=rng())
    assert torch.equal(r.h, want.h) and torch.equal(r.y, want.y)
    b, plain = te.te_layernorm_bwd(dy, r.h, r.mean, r.rstd, gamma, p=p, rng=rng()), te.te_layernorm_bwd(dy, r.h, r.mean, r.rstd, gamma)
    assert torch.equal(b.dh, plain.dh) and torch.equal(b.dx, plain.dh)
    assert torch.equal(te.te_dropout(x, p, rng()), x)
    from fp8_linear_layer_amd import block
    m = block.LayerNorm(72, dropout=p, seed=1)
    xs, rs = x.clone().requires_grad_(), res.clone().requires_grad_()
    y, _ = m(xs, rs)
    y.backward(dy)
    assert torch.equal(xs.grad, rs.grad) and (xs.grad != 0).any()
