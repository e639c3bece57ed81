"""What the norm's fp8 outputs say of NaN and infinity: a group of 128 that holds a y which is not finite stands for
NaN (by its scale), every other group is bit for bit what it is without, and the next GEMM hands it on.  Which y are
not finite is read from the same call with an fp32 output."""
import pytest
import torch

te = pytest.importorskip("fp8_linear_layer_amd")
pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
E4, E5 = te.TE_DTYPE_E4M3, te.TE_DTYPE_E5M2
F8 = {E4: torch.float8_e4m3fn, E5: torch.float8_e5m2}
ROWS, COLS = 256, 640


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    te.load_library()


def randn(shape, seed, dtype, std=1.0, mean=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)


def values(q, scales, fmt, rows):
    """What the codes and scales stand for, [rows, groups, 128]."""
    v = q.view(F8[fmt]).float().reshape(rows, -1, 128)
    return v * scales[:, :rows].t()[:, :, None]


WHERE = {"nan": [(3, 5, NAN)], "minus_nan": [(3, 5, -NAN)], "inf": [(0, 0, INF), (255, 639, -INF)], "both": [(7, 130, INF), (7, 131, NAN), (128, 300, -INF)],
         "many": [(r, (37 * r) % COLS, (NAN, INF, -INF)[r % 3]) for r in range(0, ROWS, 11)]}


@pytest.mark.parametrize("where", list(WHERE))
@pytest.mark.parametrize("fmt", [E4, E5], ids=["e4m3", "e5m2"])
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("types", ["bf16", "bf16+f32", "f32", "f32+bf16"])
def test_a_group_with_what_is_not_finite_is_nan(types, pow2, fmt, where):
    dt = [dict(bf16=torch.bfloat16, f32=torch.float32)[t] for t in types.split("+")]
    x = randn((ROWS, COLS), 1, dt[0])
    res = randn((ROWS, COLS), 2, dt[1]) if len(dt) == 2 else None
    gamma = randn((COLS,), 3, torch.bfloat16, 0.1, 1.0)
    flags = te.TE_CAST_POW2_SCALE if pow2 else 0
    clean = te.te_rmsnorm_fwd(x, gamma, residual=res, out_dtype=fmt, flags=flags, transpose=True)
    bad_rows = sorted({r for r, _, _ in WHERE[where]})
    target = x if res is None else res
    for r, c, v in WHERE[where]:
        target[r, c] = v
    y = te.te_rmsnorm_fwd(x, gamma, residual=res, out_dtype=te.TE_DTYPE_F32).y
    assert not y[bad_rows].isfinite().all(1).any()
    r = te.te_rmsnorm_fwd(x, gamma, residual=res, out_dtype=fmt, flags=flags, transpose=True)
    only = te.te_rmsnorm_fwd(x, gamma, residual=res, out_dtype=fmt, flags=flags, transpose=True, rowwise=False)
    assert torch.equal(r.qt, only.qt) and torch.equal(r.scales_t.view(torch.int32), only.scales_t.view(torch.int32))
    for q, s, cq, cs, v in ((r.q, r.scales, clean.q, clean.scales, y), (r.qt, r.scales_t, clean.qt, clean.scales_t, y.t())):
        n = v.shape[0]
        bad = ~v.reshape(n, -1, 128).isfinite().all(2)
        got = values(q, s, fmt, n)
        assert got[bad].isnan().all() and got[~bad].isfinite().all()
        # (beside an infinity a row is zeros, which are finite but not what the clean call has)
        touched = bad.clone()
        if q is r.q:
            touched[bad_rows] = True
        else:
            touched[:, [r_ // 128 for r_ in bad_rows]] = True
        same = ~touched
        assert torch.equal(q.reshape(n, -1, 128)[same], cq.reshape(n, -1, 128)[same])
        assert torch.equal(s[:, :n].t()[same], cs[:, :n].t()[same])


@pytest.mark.parametrize("value", [NAN, INF])
def test_gamma(value):
    x, gamma = randn((ROWS, COLS), 1, torch.bfloat16), randn((COLS,), 3, torch.bfloat16, 0.1, 1.0)
    gamma[200] = value
    r = te.te_rmsnorm_fwd(x, gamma, out_dtype=E4, transpose=True)
    got = values(r.q, r.scales, E4, ROWS)
    assert got[:, 1].isnan().all() and got[:, [0, 2, 3, 4]].isfinite().all()
    got = values(r.qt, r.scales_t, E4, COLS)
    assert got[200].isnan().all() and got[:200].isfinite().all() and got[201:].isfinite().all()


@pytest.mark.parametrize("pow2", [False, True])
def test_the_next_gemm_hands_it_on(pow2):
    """A NaN in one token is a NaN in that token's outputs and in no other's; in the weight gradient in the
    columns of its features."""
    flags, accum = (te.TE_CAST_POW2_SCALE, te.TE_ACCUM_FAST) if pow2 else (0, te.TE_ACCUM_FULL_FP32)
    x, gamma = randn((ROWS, COLS), 1, torch.bfloat16), randn((COLS,), 3, torch.bfloat16, 0.1, 1.0)
    w, dy = randn((384, COLS), 4, torch.bfloat16, 0.05), randn((ROWS, 384), 5, torch.bfloat16)
    x[17, 200] = NAN
    r = te.te_rmsnorm_fwd(x, gamma, out_dtype=E4, flags=flags, transpose=True)
    qw, sw = te.te_cast_fp8_per_token(w, E4, flags)
    y = te.te_fp8_gemm_fwd(r.q, r.scales, E4, qw, sw, E4, accum=accum)
    rest = torch.arange(ROWS, device="cuda") != 17
    assert y[17].isnan().all() and y[rest].isfinite().all()
    _, _, qd, sd = te.te_cast_fp8_per_token_transpose(dy, E5)
    dw = torch.zeros((384, COLS), device="cuda")
    te.te_fp8_wgrad_accum(qd, sd, E5, r.qt, r.scales_t, E4, dw, te.TE_ACCUM_FULL_FP32)
    assert dw.isnan().all()      # (the token's whole row of y is NaN)
