"""What the operators' binding refuses of tensors on the GPU: nothing is launched, the outputs given keep
their contents, and the message names the argument."""
import pytest
import torch

te = pytest.importorskip("fp8_linear_layer_amd")
pytestmark = pytest.mark.gpu
E4, BF, F32 = te.TE_DTYPE_E4M3, torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    te.load_library()


def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype, device="cuda")


X, G = (4, 256), (256,)
NORM = [
    ("x", lambda: te.te_rmsnorm_fwd(z(256), z(*G))), ("x", lambda: te.te_rmsnorm_fwd(z(*X, dtype=torch.float16), z(*G))),
    ("x", lambda: te.te_rmsnorm_fwd(z(256, 4).t(), z(*G))), ("x", lambda: te.te_rmsnorm_fwd(z(4, 1, 256).expand(4, 3, 256)[0], z(*G))),
    ("gamma", lambda: te.te_rmsnorm_fwd(z(*X), z(255))), ("gamma", lambda: te.te_rmsnorm_fwd(z(*X), z(*G, dtype=F32))),
    ("gamma", lambda: te.te_rmsnorm_fwd(z(*X), z(512)[::2])), ("gamma", lambda: te.te_rmsnorm_fwd(z(*X), z(*G).cpu())),
    ("residual", lambda: te.te_rmsnorm_fwd(z(*X), z(*G), residual=z(4, 255))), ("residual", lambda: te.te_rmsnorm_fwd(z(*X), z(*G), residual=z(*X).cpu())),
    ("h", lambda: te.te_rmsnorm_fwd(z(*X), z(*G), h=z(*X))), ("h", lambda: te.te_rmsnorm_fwd(z(*X), z(*G), residual=z(*X), h=z(*X, dtype=F32))),
    ("rstd", lambda: te.te_rmsnorm_fwd(z(*X), z(*G), rstd=z(3, dtype=F32))), ("rstd", lambda: te.te_rmsnorm_fwd(z(*X), z(*G), rstd=z(4))),
    ("y", lambda: te.te_rmsnorm_fwd(z(*X), z(*G), y=z(*X, dtype=F32))), ("y", lambda: te.te_rmsnorm_fwd(z(*X), z(*G), out_dtype=E4, y=z(*X))),
    ("fp8", lambda: te.te_rmsnorm_fwd(z(*X), z(*G), transpose=True)), ("out_dtype", lambda: te.te_rmsnorm_fwd(z(*X), z(*G), out_dtype=9)),
    ("128", lambda: te.te_rmsnorm_fwd(z(4, 192), z(192), out_dtype=E4)), ("128", lambda: te.te_rmsnorm_fwd(z(*X), z(*G), out_dtype=E4, transpose=True)),
    ("q", lambda: te.te_rmsnorm_fwd(z(*X), z(*G), out_dtype=E4, q=z(*X))), ("rowwise", lambda: te.te_rmsnorm_fwd(
        z(128, 256), z(*G), out_dtype=E4, rowwise=False, transpose=True, q=z(128, 256, dtype=torch.uint8))),
    ("scales", lambda: te.te_rmsnorm_fwd(z(*X), z(*G), out_dtype=E4, scales=z(2, 3, dtype=F32))),
    ("at least one", lambda: te.te_rmsnorm_fwd(z(*X), z(*G), out_dtype=E4, rowwise=False)), ("eps", lambda: te.te_rmsnorm_fwd(z(*X), z(*G), -1.0)),
    ("flag", lambda: te.te_rmsnorm_fwd(z(*X), z(*G), out_dtype=E4, flags=64)), ("cols", lambda: te.te_rmsnorm_fwd(z(2, 32769), z(32769))),
    ("dy", lambda: te.te_rmsnorm_bwd(z(4, 255), z(*X), z(4, dtype=F32), z(*G))), ("dres", lambda: te.te_rmsnorm_bwd(
        z(*X), z(*X), z(4, dtype=F32), z(*G), dres=z(*X, dtype=F32))),
    ("rstd", lambda: te.te_rmsnorm_bwd(z(*X), z(*X), z(4), z(*G))), ("dh", lambda: te.te_rmsnorm_bwd(z(*X), z(*X), z(4, dtype=F32), z(*G), dh=z(2, 256))),
    ("dgamma", lambda: te.te_rmsnorm_bwd(z(*X), z(*X), z(4, dtype=F32), z(*G), dgamma=z(*G))),
    ("dgamma", lambda: te.te_rmsnorm_bwd(z(*X), z(*X), z(4, dtype=F32), z(*G), dgamma=z(*G, dtype=F32), need_dgamma=False)),
    ("workspace", lambda: te.te_rmsnorm_bwd(z(*X), z(*X), z(4, dtype=F32), z(*G), workspace=z(16, dtype=torch.uint8))),
]
I32 = torch.int32
ROUTER = [
    ("logits", lambda: te.te_moe_router_fwd(z(8), 1)), ("logits", lambda: te.te_moe_router_fwd(z(4, 8, dtype=torch.float64), 1)),
    ("top_k", lambda: te.te_moe_router_fwd(z(4, 8), 0)), ("top_k", lambda: te.te_moe_router_fwd(z(4, 8), 9)), ("top_k", lambda: te.te_moe_router_fwd(z(4, 40), 17)),
    ("experts", lambda: te.te_moe_router_fwd(z(4, 2049), 1)), ("token_mask", lambda: te.te_moe_router_fwd(z(4, 8), 1, token_mask=z(3, dtype=torch.bool))),
    ("token_mask", lambda: te.te_moe_router_fwd(z(4, 8), 1, token_mask=z(4, dtype=I32))),
    ("workspace", lambda: te.te_moe_router_fwd(z(9000, 64), 1, loss=True, workspace=z(8, dtype=torch.uint8))),
    ("index", lambda: te.te_moe_router_bwd(z(4, 8), z(4, 2, dtype=torch.int64), z(4, dtype=F32))),
    ("index", lambda: te.te_moe_router_bwd(z(4, 8), z(3, 2, dtype=I32), z(4, dtype=F32))),
    ("lse", lambda: te.te_moe_router_bwd(z(4, 8), z(4, 2, dtype=I32), z(3, dtype=F32))),
    ("d_weight", lambda: te.te_moe_router_bwd(z(4, 8), z(4, 2, dtype=I32), z(4, dtype=F32), d_weight=z(4, 2))),
    ("counts", lambda: te.te_moe_router_bwd(z(4, 8), z(4, 2, dtype=I32), z(4, dtype=F32), d_loss=z(1, dtype=F32))),
    ("routed", lambda: te.te_moe_router_bwd(z(4, 8), z(4, 2, dtype=I32), z(4, dtype=F32), counts=z(8, dtype=I32), routed=z(2, dtype=I32), d_loss=z(1, dtype=F32))),
    ("d_loss", lambda: te.te_moe_router_bwd(z(4, 8), z(4, 2, dtype=I32), z(4, dtype=F32), counts=z(8, dtype=I32), routed=z(1, dtype=I32), d_loss=z(2, dtype=F32))),
    ("d_logits", lambda: te.te_moe_router_bwd(z(4, 8), z(4, 2, dtype=I32), z(4, dtype=F32), d_logits=z(4, 8, dtype=F32))),
]
CLIP = [
    ("gradients", lambda: te.te_grad_norm_clip([z(3)], 1.0, out=[])), ("gradient 1", lambda: te.te_grad_norm_clip([z(3), z(3).cpu()], 1.0)),
    ("gradient 0", lambda: te.te_grad_norm_clip([z(3, dtype=torch.float16)], 1.0)), ("gradient 0", lambda: te.te_grad_norm_clip([z(3)], 1.0, out=[z(4)])),
    ("gradient 0", lambda: te.te_grad_norm_clip([z(3)], 1.0, out=[None])), ("max_norm", lambda: te.te_grad_norm_clip([z(3)], 0.0)),
    ("norm", lambda: te.te_grad_norm_clip([z(3)], 1.0, norm=z(1))), ("workspace", lambda: te.te_grad_norm_clip([z(3)], 1.0, workspace=z(8, dtype=torch.uint8))),
]


@pytest.mark.parametrize("what,call", NORM + ROUTER + CLIP)
def test_refused(what, call):
    with pytest.raises(te.TeFp8Error, match=what):
        call()
    torch.cuda.synchronize()


def test_a_refused_call_leaves_its_outputs():
    y, rstd = torch.full((4, 256), 5.0, dtype=BF, device="cuda"), torch.full((4,), 5.0, device="cuda")
    with pytest.raises(te.TeFp8Error):
        te.te_rmsnorm_fwd(z(*X), z(255), y=y, rstd=rstd)
    g = [torch.full((3,), 5.0, device="cuda"), z(3, dtype=torch.float16)]
    with pytest.raises(te.TeFp8Error):
        te.te_grad_norm_clip(g, 0.1)
    assert (y == 5).all() and (rstd == 5).all() and (g[0] == 5).all()
    with pytest.raises(TypeError):
        te.te_rmsnorm_fwd(z(*X), z(*G), eps="small")
