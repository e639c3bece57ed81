"""A gated block's operators at the ends of what they take: the longest contraction and the most features, row strides just
below 64 MiB, more rows than one launch has, the longest rows in the transposed layout; and the gated modules without a graph.

Tolerances: those of test_gpu_gated and test_gpu_layernorm."""
import gc

import numpy as np
import pytest
import torch

import oracle
from parity import host, shost
from test_gpu_gated import E4, E5, F32, SILU, U, close, dgrad64, forward64, gen, operand
from test_gpu_layernorm import EPS, check_fwd, normal, vector

te = pytest.importorskip("fp8_linear_layer_amd")
pytestmark = pytest.mark.gpu
MOST = 1 << 22


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    te.load_library()
    # (what the products' library keeps for itself is allocated now, not inside one of the gigabytes that follow, which
    # could then not be given back)
    one = torch.ones((64, 64), dtype=torch.float64, device="cuda")
    torch.cuda.synchronize()
    one @ one
    yield
    gc.collect()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("rows", [1, 130])
def test_the_longest_contraction(rows):
    g, hidden = gen(rows), 128
    x, sx = operand(g, rows, MOST, E4)
    w, sw = operand(g, 2 * hidden, MOST, E4, MOST ** -0.5)
    z, ez, y, bound = forward64(x, sx, E4, w, sw, E4, SILU, rows <= 128)
    r = te.te_fp8_gated_fwd(x, sx, E4, w, sw, E4, out_dtype=F32, need_z=True)
    close(r.z, z, ez + 2.0 ** -8 * (z.abs() + ez), "z")
    close(r.y, y, bound + U * y.abs(), "y")
    dz, e = dgrad64(x, sx, E4, w[:hidden], sw[:, :hidden], E4, r.z, SILU)
    d = te.te_fp8_gated_dgrad(x, sx, E4, w[:hidden], sw[:, :hidden].contiguous(), E4, r.z, out_dtype=F32)
    close(d.dz, dz, e + U * dz.abs(), "dz")


@pytest.mark.parametrize("rows", [1, 40, 130])
def test_the_most_features(rows):
    g, k, n = gen(rows), 128, 4096
    x, sx = operand(g, rows, k, E4)
    w, sw = operand(g, 2 * MOST, k, E4, k ** -0.5)
    r = te.te_fp8_gated_fwd(x, sx, E4, w, sw, E4, out_dtype=F32, need_z=True)
    c = te.te_fp8_gated_fwd(x, sx, E4, w, sw, E4, out_dtype=E4)
    wt, swt = w[:MOST], sw[:, :MOST].contiguous()
    d = te.te_fp8_gated_dgrad(x, sx, E4, wt, swt, E4, r.z, out_dtype=F32)
    for f in (0, MOST // 2, MOST - n):       # (n features at a time in 64 bits)
        z, ez, y, bound = forward64(x, sx, E4, w[2 * f:2 * (f + n)], sw[:, 2 * f:2 * (f + n)], E4, SILU, rows <= 128)
        close(r.z[:, 2 * f:2 * (f + n)], z, ez + 2.0 ** -8 * (z.abs() + ez), "z")
        close(r.y[:, f:f + n], y, bound + U * y.abs(), "y")
        oq, os_ = oracle.cast_per_token_f32(host(r.y[:, f:f + n].contiguous()).numpy(), oracle.E4M3, False)
        assert np.array_equal(host(c.q[:, f:f + n].contiguous()).numpy(), oq)
        assert np.array_equal(shost(c.scales[f // 128:(f + n) // 128].contiguous(), rows).view(np.uint32), os_.view(np.uint32))
        dz, e = dgrad64(x, sx, E4, wt[f:f + n], swt[:, f:f + n], E4, r.z[:, 2 * f:2 * (f + n)], SILU)
        close(d.dz[:, 2 * f:2 * (f + n)], dz, e + U * dz.abs(), "dz")


@pytest.mark.parametrize("rows", [65, 130, 1300])
def test_row_strides_just_below_64_mib(rows):
    g, k, hidden = gen(rows), 128, 256
    x, sx = operand(g, rows, k, E4)
    w, sw = operand(g, 2 * hidden, k, E4, k ** -0.5)
    wt, swt = w[:hidden], sw[:, :hidden].contiguous()
    want = te.te_fp8_gated_fwd(x, sx, E4, w, sw, E4, need_z=True)
    dz = te.te_fp8_gated_dgrad(x, sx, E4, wt, swt, E4, want.z).dz
    ld = (1 << 25) - 8
    buf = torch.full((rows * ld,), 7, dtype=torch.bfloat16, device="cuda")

    def wide(cols, first):
        return buf[first:].as_strided((rows, cols), (ld, 1))

    y, z, out = wide(hidden, 1024), wide(2 * hidden, 4096), wide(2 * hidden, 8192)
    te.te_fp8_gated_fwd(x, sx, E4, w, sw, E4, y=y, z=z)
    assert torch.equal(y, want.y) and torch.equal(z, want.z)
    te.te_fp8_gated_dgrad(x, sx, E4, wt, swt, E4, z, dz=out)
    assert torch.equal(out, dz)
    assert (wide(1024, 0) == 7).all() and (wide(2048, 1024 + hidden) == 7).all() and (wide(2048, 4096 + 2 * hidden) == 7).all()
    assert (wide(2048, 8192 + 2 * hidden) == 7).all()
    if rows % 128 == 2:     # both casts, of whole groups of rows
        rows, x, sx, z = rows - 2, x[:-2], sx[:, :rows - 2].contiguous(), z[:-2]
        both = dict(out_dtype=E5, transpose=True)
        a, b = te.te_fp8_gated_dgrad(x, sx, E4, wt, swt, E4, z, **both), te.te_fp8_gated_dgrad(x, sx, E4, wt, swt, E4, want.z[:-2].contiguous(), **both)
        assert torch.equal(a.q, b.q) and torch.equal(a.qt, b.qt) and torch.equal(a.scales, b.scales) and torch.equal(a.scales_t, b.scales_t)
    for bad in (1 << 25, (1 << 25) + 8):
        with pytest.raises(te.TeFp8Error, match="64 MiB"):
            te.te_fp8_gated_fwd(x[:2], sx[:, :4].contiguous(), E4, w, sw, E4, y=buf.as_strided((2, hidden), (bad, 1)))


def test_norm_of_more_rows_than_a_launch_has():
    rows, cols = (1 << 27) + 37, 17
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=g)
    gamma, beta = vector(g, cols, 0.1, 1.0), vector(g, cols, 0.3)
    r = te.te_layernorm_fwd(x, gamma, beta, EPS)
    b = te.te_layernorm_bwd(x, x, r.mean, r.rstd, gamma, need_dgamma=False, need_dbeta=False)
    for first in (0, (1 << 27) - 50, rows - 100):
        at = slice(first, first + 100)
        few = te.te_layernorm_fwd(x[at], gamma, beta, EPS)
        check_fwd(x[at], None, 0.0, gamma, beta, few)
        assert torch.equal(few.y, r.y[at]) and torch.equal(few.mean, r.mean[at]) and torch.equal(few.rstd, r.rstd[at])
        d = te.te_layernorm_bwd(x[at], x[at], few.mean, few.rstd, gamma, need_dgamma=False, need_dbeta=False)
        assert torch.equal(d.dh, b.dh[at])


@pytest.mark.parametrize("cols", [16392, 32768])
def test_transposed_cast_of_the_longest_rows(cols):
    g = torch.Generator(device="cuda").manual_seed(cols)
    x, res = normal(g, (256, cols), torch.bfloat16), normal(g, (256, cols), torch.bfloat16, 2.0)
    gamma, beta = vector(g, cols, 0.1, 1.0), vector(g, cols, 0.3)
    y32 = host(te.te_layernorm_fwd(x, gamma, beta, EPS, residual=res, out_dtype=F32).y).numpy()
    r = te.te_layernorm_fwd(x, gamma, beta, EPS, residual=res, out_dtype=E4, rowwise=cols % 128 == 0, transpose=True)
    for q, s, y, n in ((r.q, r.scales, y32, 256), (r.qt, r.scales_t, np.ascontiguousarray(y32.T), cols)):
        if q is not None:
            oq, os_ = oracle.cast_per_token_f32(y, oracle.E4M3, False)
            assert np.array_equal(host(q).numpy(), oq) and np.array_equal(shost(s, n).view(np.uint32), os_.view(np.uint32))


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
@pytest.mark.parametrize("training", [True, False])
def test_modules_without_a_graph(mode, training):
    """The forward pass of a module that records no graph is the one that does."""
    from fp8_linear_layer_amd import block, linear
    T, K = 256, 256
    g = torch.Generator(device="cuda").manual_seed(0)
    x, res = normal(g, (T, K), torch.bfloat16), normal(g, (T, K), torch.bfloat16)
    m, n = linear.Fp8GatedMlp(K, 512, generator=g), block.Fp8NormGatedMlp(K, 512, dropout=0.3, seed=5, generator=g).train(training)
    state = n.draw()
    want = m(x).detach(), *(t.detach() for t in n(x, res, state)), n(x)[0].detach()
    with mode():
        got = m(x), *n(x, res, state), n(x)[0]
    assert all(torch.equal(a, b) and not b.requires_grad for a, b in zip(want, got))
    y, h = n(x, res, state)      # and the graph of a later one is whole
    (y.float().sum() + h.float().sum()).backward()
    assert (n.w1.main_grad != 0).any() and (n.weight.main_grad != 0).any()
