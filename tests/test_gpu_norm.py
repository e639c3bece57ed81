"""GPU parity of te_rmsnorm_fwd / te_rmsnorm_bwd with the formulas in 64 bits.

Tolerances (u = 2^-24, the rounding of fp32): the sum of squares has only positive terms and at most
64 additions in a row, so rstd is within (64 / 2 + 4) u of its exact value, and y, two products on, within
40 u; a stored bf16 value is off by half a step more (2^-8 of the value), fp32 by u.  The fp8 outputs
are exactly the cast (the oracle's, in fp32) of the y that the same call stores in fp32, and within half a
code step and those 40 u of the 64-bit y."""
import numpy as np
import pytest
import torch

import oracle
from parity import host, shost

te = pytest.importorskip("fp8_linear_layer_amd")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
OUT = {"bf16": te.TE_DTYPE_BF16, "f32": te.TE_DTYPE_F32, "e4m3": te.TE_DTYPE_E4M3, "e5m2": te.TE_DTYPE_E5M2}
FMT = {"e4m3": oracle.E4M3, "e5m2": oracle.E5M2}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
# half a code step relative to the value, and half the step of the subnormals at scale 1
F8_HALF = {"e4m3": (2.0 ** -4, 2.0 ** -10), "e5m2": (2.0 ** -3, 2.0 ** -17)}
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    te.load_library()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, shape, dtype, std=1.0, mean=0.0, ld=None, shift=0):
    """A matrix inside a larger buffer: row stride ld, first element `shift` elements in."""
    rows, cols = shape
    ld = ld or cols
    buf = torch.full((rows * ld + shift + 16,), float("nan"), dtype=dtype, device="cuda")
    view = buf[shift:].as_strided((rows, cols), (ld, 1))
    view.copy_(torch.randn(shape, generator=g, device="cuda") * std + mean)
    return view


def padded(shape, dtype, ld, shift=0, fill=7):
    rows, cols = shape
    buf = torch.full((rows * ld + shift + 32,), fill, dtype=dtype, device="cuda")
    return buf, buf[shift:].as_strided((rows, cols), (ld, 1))


def assert_untouched(buf, view, fill=7):
    """Everything of the buffer outside the view still holds the fill value."""
    keep = torch.ones(buf.shape, dtype=torch.bool, device="cuda")
    keep.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(False)
    assert (buf[keep] == fill).all()


def exact_fwd(v, gamma):
    v = v.double()
    rstd = 1.0 / torch.sqrt((v * v).mean(1) + EPS)
    return rstd, v * rstd[:, None] * gamma.double()


def close(got, want, rel, floor=0.0, what=""):
    err = (got.double() - want).abs()
    bad = ~(err <= want.abs() * rel + floor)
    assert not bad.any(), f"{what}: {int(bad.sum())} off, worst {float((err / (want.abs() * rel + floor + 1e-300)).max()):.3g} of the bound"


def check_fwd(x, res, gamma, r):
    if res is not None:
        s = x.double() + res.double()
        close(r.h, s, HALF[r.h.dtype] + 2 * U, what="h")
        v = r.h
    else:
        v = x
    rstd, y = exact_fwd(v, gamma)
    close(r.rstd, rstd, 36 * U, what="rstd")
    return y


COLS = [1, 2, 7, 8, 9, 15, 64, 129, 250, 256, 257, 512, 513, 1000, 2048, 2056, 2112, 4096, 4097, 7168, 8192, 8200, 14336, 16384, 16392, 20003, 32768]


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("xt,ht,out", [("bf16", "bf16", "bf16"), ("bf16", "f32", "f32"), ("f32", "", "bf16"),
                                       ("f32", "bf16", "f32"), ("bf16", "", "f32"), ("f32", "f32", "bf16")])
def test_forward(cols, xt, ht, out):
    for rows in (1, 5, 131):
        g = gen(cols * 7 + rows)
        x = normal(g, (rows, cols), DT[xt], 0.7)
        res = normal(g, (rows, cols), DT[ht], 2.0) if ht else None
        gamma = normal(g, (1, cols), torch.bfloat16, 0.1, 1.0)[0]
        r = te.te_rmsnorm_fwd(x, gamma, EPS, residual=res, out_dtype=OUT[out])
        y = check_fwd(x, res, gamma, r)
        close(r.y, y, HALF[DT[out]] + 40 * U, what="y")
        again = te.te_rmsnorm_fwd(x, gamma, EPS, residual=res, out_dtype=OUT[out])
        assert torch.equal(again.y, r.y) and torch.equal(again.rstd, r.rstd)


@pytest.mark.parametrize("rows,cols", [(1, 128), (3, 256), (128, 128), (130, 640), (77, 2176), (33, 4096), (256, 7168), (9, 14336),
                                       (2, 32768), (1000, 384)])
@pytest.mark.parametrize("out", ["e4m3", "e5m2"])
@pytest.mark.parametrize("xt,ht,pow2", [("bf16", "bf16", False), ("f32", "", True), ("bf16", "f32", False), ("f32", "bf16", True)])
def test_forward_fp8(rows, cols, out, xt, ht, pow2):
    g = gen(rows * 31 + cols)
    x = normal(g, (rows, cols), DT[xt], 0.7)
    res = normal(g, (rows, cols), DT[ht], 2.0) if ht else None
    gamma = normal(g, (1, cols), torch.bfloat16, 0.1, 1.0)[0]
    x[:, :128] = 0          # a group of zeros
    if res is not None:
        res[:, :128] = 0
    flags = te.TE_CAST_POW2_SCALE if pow2 else 0
    both = rows % 128 == 0
    r = te.te_rmsnorm_fwd(x, gamma, EPS, residual=res, out_dtype=OUT[out], flags=flags, transpose=both)
    y64 = check_fwd(x, res, gamma, r)
    plain = te.te_rmsnorm_fwd(x, gamma, EPS, residual=res, out_dtype=te.TE_DTYPE_F32)
    assert torch.equal(plain.rstd, r.rstd)
    y32 = host(plain.y).numpy()
    for q, s, y, n in [(r.q, r.scales, y32, rows)] + ([(r.qt, r.scales_t, np.ascontiguousarray(y32.T), cols)] if both else []):
        oq, os_ = oracle.cast_per_token_f32(y, FMT[out], pow2)
        assert np.array_equal(host(q).numpy(), oq)
        assert np.array_equal(shost(s, n).view(np.uint32), os_.view(np.uint32))
    scale = r.scales[:, :rows].t().double().repeat_interleave(128, 1)
    rel, sub = F8_HALF[out]
    err = (r.q.view(F8[out]).double() * scale - y64).abs()
    assert (err <= y64.abs() * (rel + 44 * U) + scale * sub).all()
    if both:      # the transposed output alone gives the same bytes
        t = te.te_rmsnorm_fwd(x, gamma, EPS, residual=res, out_dtype=OUT[out], flags=flags, rowwise=False, transpose=True)
        assert t.q is None and torch.equal(t.qt, r.qt) and torch.equal(t.scales_t, r.scales_t)
        assert torch.equal(t.rstd, r.rstd) and (res is None or torch.equal(t.h, r.h))


@pytest.mark.parametrize("xt", ["bf16", "f32"])
def test_transposed_cast_of_columns_that_fill_no_tile(xt):
    rows, cols = 256, 328
    g = gen(5)
    x = normal(g, (rows, cols), DT[xt])
    gamma = normal(g, (1, cols), torch.bfloat16, 0.1, 1.0)[0]
    r = te.te_rmsnorm_fwd(x, gamma, EPS, out_dtype=OUT["e4m3"], rowwise=False, transpose=True)
    y32 = host(te.te_rmsnorm_fwd(x, gamma, EPS, out_dtype=te.TE_DTYPE_F32).y).numpy()
    oq, os_ = oracle.cast_per_token_f32(np.ascontiguousarray(y32.T), oracle.E4M3, False)
    assert np.array_equal(host(r.qt).numpy(), oq) and np.array_equal(shost(r.scales_t, cols).view(np.uint32), os_.view(np.uint32))


@pytest.mark.parametrize("cols,ldx,ldr,ldh,ldy,shift", [(250, 251, 259, 250, 253, 1), (2112, 2115, 2112, 2113, 2200, 3), (9, 9, 11, 13, 9, 1),
                                                        (4096, 4100, 4097, 4096, 4099, 5), (5, 6, 7, 8, 9, 1)])
@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_forward_strides_and_alignment(cols, ldx, ldr, ldh, ldy, shift, t):
    rows = 37
    g = gen(cols)
    x = normal(g, (rows, cols), DT[t], ld=ldx, shift=shift)
    res = normal(g, (rows, cols), DT[t], 2.0, ld=ldr, shift=shift + 1)
    gamma = normal(g, (1, cols), torch.bfloat16, 0.1, 1.0, shift=1)[0]
    hb, h = padded((rows, cols), DT[t], ldh, shift)
    yb, y = padded((rows, cols), DT[t], ldy, shift + 2)
    r = te.te_rmsnorm_fwd(x, gamma, EPS, residual=res, out_dtype=OUT[t], h=h, y=y)
    want = check_fwd(x, res, gamma, r)
    close(y, want, HALF[DT[t]] + 40 * U, what="y")
    assert_untouched(hb, h)
    assert_untouched(yb, y)


@pytest.mark.parametrize("cols", [3, 61, 2051, 4096])
def test_residual_in_place(cols):
    g = gen(cols)
    x, res = normal(g, (70, cols), torch.bfloat16), normal(g, (70, cols), torch.bfloat16, 2.0)
    gamma = normal(g, (1, cols), torch.bfloat16, 0.1, 1.0)[0]
    want = te.te_rmsnorm_fwd(x, gamma, EPS, residual=res)
    got = te.te_rmsnorm_fwd(x, gamma, EPS, residual=res, h=res)
    assert got.h is res and torch.equal(res, want.h) and torch.equal(got.y, want.y)


def test_special_values():
    cols = 256
    x = torch.zeros((6, cols), dtype=torch.float32, device="cuda")
    x[1, 3] = float("nan")
    x[2, 5] = float("inf")
    x[3] = 1e-30                       # squares below fp32's range
    x[4, 0] = -0.0
    x[5] = 3.0
    gamma = torch.ones((cols,), dtype=torch.bfloat16, device="cuda")
    r = te.te_rmsnorm_fwd(x, gamma, EPS, out_dtype=te.TE_DTYPE_F32)
    assert (r.y[0] == 0).all() and torch.allclose(r.rstd[0], torch.tensor(EPS ** -0.5, device="cuda"))
    assert r.y[1].isnan().all()
    assert r.rstd[2] == 0 and r.y[2, 5].isnan() and (r.y[2, :5] == 0).all()
    close(r.y[3], x[3].double() * EPS ** -0.5, 40 * U)
    close(r.y[5], torch.full((cols,), 3.0 / (9.0 + EPS) ** 0.5, dtype=torch.float64, device="cuda"), 40 * U)


# ------------------------------------------------------------ backward
def exact_bwd(dy, h, rstd, gamma, dres):
    dy, h, r, gm = dy.double(), h.double(), rstd.double()[:, None], gamma.double()
    xh, g = h * r, dy * gm
    mean = (g * xh).mean(1, keepdim=True)
    dh = r * (g - xh * mean)
    mag = r * (g.abs() + xh.abs() * (g * xh).abs().mean(1, keepdim=True))
    if dres is not None:
        dh, mag = dh + dres.double(), mag + dres.double().abs()
    return dh, mag, (dy * xh).sum(0), (dy * xh).abs().sum(0)


def check_bwd(dy, h, rstd, gamma, dres, dh, dgamma):
    """The row's mean has at most 64 additions in a row of terms of three roundings each, and dh adds six
    roundings; a column's sum takes its rows in at most rows / 256 + 64 additions."""
    want, mag, dg, dgmag = exact_bwd(dy, h, rstd, gamma, dres)
    err = (dh.double() - want).abs()
    assert (err <= 80 * U * mag + HALF[dh.dtype] * want.abs()).all(), f"dh off by {float((err / (mag + 1e-300)).max() / U):.1f} u of its terms"
    err = (dgamma.double() - dg).abs()
    assert (err <= (dy.shape[0] / 256 + 72) * U * dgmag).all(), "dgamma"


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("yt,ht,res", [("bf16", "bf16", True), ("f32", "f32", True), ("bf16", "f32", False), ("f32", "bf16", False)])
def test_backward(cols, yt, ht, res):
    for rows in (1, 3, 131) + ((2500,) if cols <= 2112 else ()):
        g = gen(cols * 5 + rows)
        h = normal(g, (rows, cols), DT[ht], 1.5)
        rstd = torch.rsqrt(h.double().square().mean(1) + EPS).float()
        dy = normal(g, (rows, cols), DT[yt], 1e-3)
        dres = normal(g, (rows, cols), DT[ht], 1e-3) if res else None
        gamma = normal(g, (1, cols), torch.bfloat16, 0.1, 1.0)[0]
        dh, dgamma = te.te_rmsnorm_bwd(dy, h, rstd, gamma, dres=dres)
        check_bwd(dy, h, rstd, gamma, dres, dh, dgamma)
        dh2, dgamma2 = te.te_rmsnorm_bwd(dy, h, rstd, gamma, dres=dres)
        assert torch.equal(dh, dh2) and torch.equal(dgamma, dgamma2)
        dh3, none = te.te_rmsnorm_bwd(dy, h, rstd, gamma, dres=dres, need_dgamma=False)
        assert none is None and torch.equal(dh, dh3)


@pytest.mark.parametrize("cols,ld,shift", [(250, 253, 1), (2112, 2117, 3), (5, 7, 1), (4096, 4099, 5), (20003, 20011, 1), (32768, 32768, 0)])
@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_backward_strides_and_in_place(cols, ld, shift, t):
    rows = 41
    g = gen(cols + ld)
    h = normal(g, (rows, cols), DT[t], 1.5, ld=ld, shift=shift)
    rstd = torch.rsqrt(h.double().square().mean(1) + EPS).float()
    dy = normal(g, (rows, cols), DT[t], 1e-3, ld=ld + 1, shift=shift + 1)
    gamma = normal(g, (1, cols), torch.bfloat16, 0.1, 1.0, shift=1)[0]
    buf, dres = padded((rows, cols), DT[t], ld + 2, shift)
    dres.copy_(normal(g, (rows, cols), DT[t], 1e-3))
    before = dres.clone()
    dh, dgamma = te.te_rmsnorm_bwd(dy, h, rstd, gamma, dres=dres, dh=dres)
    assert dh is dres
    check_bwd(dy, h, rstd, gamma, before, dh, dgamma)
    assert_untouched(buf, dres)


@pytest.mark.parametrize("ht", ["bf16", "f32"])
def test_backward_against_differences(ht):
    """The derivative of L(h) = sum(y * dy) along a direction, from the forward kernel's fp32 outputs at
    h +- step * d.  The outputs' rounding adds at most 40 u of sum |y dy| / step; the differences' own error is
    that of the same differences in 64 bits."""
    rows, cols, step = 12, 320, 2.0 ** -5
    g = gen(11)
    d = torch.randint(-4, 5, (rows, cols), generator=g, device="cuda").float() / 4
    h = (torch.randint(-64, 65, (rows, cols), generator=g, device="cuda") / 32).to(DT[ht])
    gamma = normal(g, (1, cols), torch.bfloat16, 0.1, 1.0)[0]
    dy = normal(g, (rows, cols), torch.float32)
    r = te.te_rmsnorm_fwd(h, gamma, EPS, out_dtype=te.TE_DTYPE_F32)
    dh, dgamma = te.te_rmsnorm_bwd(dy, h, r.rstd, gamma)

    def value(at, kernel):
        if not kernel:
            return (exact_fwd(at, gamma)[1] * dy.double()).sum(1)
        return (te.te_rmsnorm_fwd(at, gamma, EPS, out_dtype=te.TE_DTYPE_F32).y.double() * dy.double()).sum(1)

    up, down = (h.float() + step * d).to(DT[ht]), (h.float() - step * d).to(DT[ht])
    d = (up.double() - down.double()) / (2 * step)      # the direction between the points as they are stored
    diff = (value(up, True) - value(down, True)) / (2 * step)
    diff64 = (value(up, False) - value(down, False)) / (2 * step)
    want64, mag, _, _ = exact_bwd(dy, h, r.rstd, gamma, None)
    along = (dh.double() * d.double()).sum(1)
    tol = 40 * U * (r.y.double() * dy.double()).abs().sum(1) / step + (diff64 - (want64 * d.double()).sum(1)).abs()
    tol += ((80 * U * mag + HALF[dh.dtype] * want64.abs()) * d.double().abs()).sum(1)
    assert ((along - diff).abs() <= tol).all()


# ------------------------------------------------------------ both
def test_no_rows():
    gamma = torch.ones((256,), dtype=torch.bfloat16, device="cuda")
    x = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    r = te.te_rmsnorm_fwd(x, gamma, residual=x, out_dtype=te.TE_DTYPE_E4M3, transpose=True)
    assert r.q.shape == (0, 256) and r.qt.shape == (256, 0)
    dh, dgamma = te.te_rmsnorm_bwd(x, x, r.rstd, gamma, dgamma=torch.full((256,), 9.0, device="cuda"))
    assert dh.shape == (0, 256) and (dgamma == 0).all()


def test_offsets_past_32_bits():
    rows, cols, ld = 3, 520, 1 << 31
    big = torch.empty((2 * ld + cols,), dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((rows, cols), (ld, 1))
    g = gen(3)
    x.copy_(torch.randn((rows, cols), generator=g, device="cuda"))
    gamma = normal(g, (1, cols), torch.bfloat16, 0.1, 1.0)[0]
    small = x.clone()
    a, b = te.te_rmsnorm_fwd(x, gamma), te.te_rmsnorm_fwd(small, gamma)
    assert torch.equal(a.y, b.y)
    da, ga = te.te_rmsnorm_bwd(small, x, a.rstd, gamma)
    db, gb = te.te_rmsnorm_bwd(small, small, a.rstd, gamma)
    assert torch.equal(da, db) and torch.equal(ga, gb)


def test_more_rows_than_one_launch_holds():
    """2^28 rows of one column at sixteen threads each pass the threads of a launch."""
    rows = (1 << 28) + 77
    x = torch.full((rows, 1), 2.0, dtype=torch.bfloat16, device="cuda")
    x[-1], x[(1 << 27) + 5] = 0.5, -4.0
    gamma = torch.full((1,), 3.0, dtype=torch.bfloat16, device="cuda")
    r = te.te_rmsnorm_fwd(x, gamma, 0.0)
    assert float(r.rstd[-1]) == 2.0 and float(r.rstd[(1 << 27) + 5]) == 0.25 and int((r.rstd == 0.5).sum()) == rows - 2
    assert float(r.y[(1 << 27) + 5]) == -3.0 and int((r.y == 3.0).sum()) == rows - 1


@pytest.mark.parametrize("rows,cols,ld,xt,ht", [(40000, 2049, 2051, "bf16", ""), (20000, 1030, 1033, "f32", "bf16"), (17000, 4096, 4096, "bf16", "f32"),
                                                (9 << 20, 9, 9, "bf16", "")])
def test_inputs_larger_than_the_caches(rows, cols, ld, xt, ht):
    """Read past the caches (128 MiB and more), at odd lengths and strides."""
    g = gen(cols)
    x = normal(g, (rows, cols), DT[xt], 0.7, ld=ld, shift=1)
    res = normal(g, (rows, cols), DT[ht], 2.0, ld=ld, shift=3) if ht else None
    gamma = normal(g, (1, cols), torch.bfloat16, 0.1, 1.0)[0]
    r = te.te_rmsnorm_fwd(x, gamma, EPS, residual=res)
    y = check_fwd(x, res, gamma, r)
    close(r.y, y, HALF[torch.bfloat16] + 40 * U, what="y")


def test_given_stream_owns_what_the_call_allocates():
    x = normal(gen(1), (512, 1024), torch.bfloat16)
    gamma = normal(gen(2), (1, 1024), torch.bfloat16, 0.1, 1.0)[0]
    want = te.te_rmsnorm_fwd(x, gamma)
    dwant = te.te_rmsnorm_bwd(x, x, want.rstd, gamma)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    before = torch.cuda.current_stream()
    for _ in range(20):      # (workspaces and outputs come and go on both streams)
        got = te.te_rmsnorm_fwd(x, gamma, stream=side)
        dgot = te.te_rmsnorm_bwd(x, x, got.rstd, gamma, stream=side)
        noise = [torch.full_like(x, float("nan")) for _ in range(4)]
        assert torch.cuda.current_stream() == before
    side.synchronize()
    del noise
    assert torch.equal(got.y, want.y) and all(torch.equal(a, b) for a, b in zip(dgot, dwant))


def test_other_stream_and_graph():
    rows, cols = 256, 1024
    g = gen(21)
    x, res = normal(g, (rows, cols), torch.bfloat16), normal(g, (rows, cols), torch.bfloat16, 2.0)
    gamma = normal(g, (1, cols), torch.bfloat16, 0.1, 1.0)[0]
    dy = normal(g, (rows, cols), torch.bfloat16, 1e-3)

    def step(stream=None):
        r = te.te_rmsnorm_fwd(x, gamma, EPS, residual=res, out_dtype=te.TE_DTYPE_E4M3, transpose=True, stream=stream)
        dh, dg = te.te_rmsnorm_bwd(dy, r.h, r.rstd, gamma, dres=dy, stream=stream)
        return [r.h, r.rstd, r.q, r.scales, r.qt, r.scales_t, dh, dg]

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
        x.copy_(torch.randn((rows, cols), generator=gen(100 + i), device="cuda"))
        graph.replay()
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager)), i
