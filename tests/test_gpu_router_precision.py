"""The row sum of the router's softmax is an fp32 result: rows of one logit and 2047 others that stand x below it and
share their value, so that the errors of their exponentials do not average out.  The chosen expert's weight is
1 / (1 + 2047 exp(x)), of which the 2047 have about half the sum at x = -7.6.

Its error over many x, in u = 2^-24: an addition is off by at most half of its last place, 0.42 u of the sum rms.
Added in pairs, the equal terms double exactly, and only the 11 partial sums that the large logit is in are rounded:
0.42 u of 1, 1, ... 1.25, 1.5, 2 out of 2, together 0.9 u; the exponential and its correction 1 u of the half that they
make, and the division and the store 0.4 u: 1.1 u rms.  1.5 u is allowed.  (A product x log2(e) rounded to fp32 alone,
8 to 16 here, makes 1.9 u; added one after the other, the terms are all rounded the same way.)"""
import pytest
import torch

te = pytest.importorskip("fp8_linear_layer_amd")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_row_sum(dtype, renorm):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    tokens, experts = 4000, 2048
    g = torch.Generator(device="cuda").manual_seed(7)
    x = (torch.rand((tokens, 1), generator=g, device="cuda") * -2.5 - 6.5).to(dtype)
    v = x.expand(tokens, experts).clone()
    at = torch.randint(0, experts, (tokens,), generator=g, device="cuda")
    v[torch.arange(tokens, device="cuda"), at] = 0.0
    total = 1.0 + (experts - 1) * x[:, 0].double().exp()
    r = te.te_moe_router_fwd(v, 2, renormalize=renorm, loss=True)
    assert torch.equal(r.index[:, 0].long(), at)
    if renorm:      # of the two chosen ones: their own sum
        total = 1.0 + x[:, 0].double().exp()
    off = (r.weight[:, 0].double() * total - 1.0) / U
    assert float(off.square().mean().sqrt()) <= 1.5, float(off.square().mean().sqrt())
    if not renorm:
        lse = (r.lse.double() - total.log()) / U       # logf and the sum's 1.1 u, at a value below 1.5
        assert float(lse.square().mean().sqrt()) <= 2.5
