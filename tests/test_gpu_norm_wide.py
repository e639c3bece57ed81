"""The norm's forward pass over 4097 to 8192 columns, whose rows have another split over threads: every type against
the formula in 64 bits, and rows of one length the same bits whatever their number.  Tolerances as for other lengths
(u = 2^-24): y within 40 u, a stored bf16 half a step (2^-8) more."""
import pytest
import torch

te = pytest.importorskip("fp8_linear_layer_amd")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    te.load_library()


@pytest.mark.parametrize("cols", [4097, 4104, 5120, 7168, 7169, 7175, 7176, 7424, 7935, 7936, 7937, 8184, 8185, 8191, 8192, 8193])
@pytest.mark.parametrize("xt,rt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32"), ("bf16", ""), ("f32", "")])
def test_forward(cols, xt, rt):
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = (torch.randn((37, cols), generator=g, device="cuda") * 0.7).to(DT[xt])
    res = (torch.randn((37, cols), generator=g, device="cuda") * 2).to(DT[rt]) if rt else None
    gamma = (torch.randn((cols,), generator=g, device="cuda") * 0.1 + 1).bfloat16()
    for out, dt in ((te.TE_DTYPE_F32, torch.float32), (te.TE_DTYPE_BF16, torch.bfloat16)):
        r = te.te_rmsnorm_fwd(x, gamma, residual=res, out_dtype=out)
        h = (x.float() + res.float()).to(res.dtype) if rt else x
        assert r.h is None or torch.equal(r.h, h)
        v = h.double()
        rstd = 1.0 / torch.sqrt(v.square().mean(1) + 1e-5)
        y = v * rstd[:, None] * gamma.double()
        assert ((r.rstd.double() - rstd).abs() <= 36 * U * rstd).all()
        assert ((r.y.double() - y).abs() <= (40 * U + (HALF[dt] if dt != torch.float32 else 0)) * y.abs()).all()
        one = te.te_rmsnorm_fwd(x[5:6], gamma, residual=None if res is None else res[5:6], out_dtype=out)
        assert torch.equal(one.y, r.y[5:6]) and torch.equal(one.rstd, r.rstd[5:6])
