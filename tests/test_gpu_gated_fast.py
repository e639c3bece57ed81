"""te_fp8_gated_fwd under TE_ACCUM_FAST at sizes where every workgroup has several tiles, on power-of-two scales, on others,
and on scales of which some tiles have a few others; and the smallest fp8 outputs of both gated calls, none of them zero.

Tolerances: those of test_gpu_gated (the bound of the products is that of either update, so it holds whichever a tile takes).
fp8 outputs are exactly the cast of the fp32 output of the same tiles."""
import pytest
import torch

from test_gpu_gated import BF, E4, E5, F32, GELU, SILU, U, check_casts, close, dgrad64, forward64, gen, operand

te = pytest.importorskip("fp8_linear_layer_amd")
pytestmark = pytest.mark.gpu
FAST = te.TE_ACCUM_FAST


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    te.load_library()


def spoil(s, at):
    """Scales that are no powers of two for the columns `at` of a block-major scale array, in one of the blocks."""
    s[s.shape[0] // 2, at] *= 1.5


@pytest.mark.parametrize("rows", [8192, 7999])
@pytest.mark.parametrize("scales", ["power of two", "other", "some rows", "some features"])
@pytest.mark.parametrize("act", [SILU, GELU])
def test_tiles(rows, scales, act):
    k, hidden = 384, 2048 + 128     # 32 x 17 tiles for 256 workgroups
    g = gen(rows + len(scales))
    pow2 = scales != "other"
    x, sx = operand(g, rows, k, E4, pow2=pow2)
    w, sw = operand(g, 2 * hidden, k, E4, 1.5 * k ** -0.5, pow2=pow2)
    if scales == "some rows":       # (tiles of rows 256 .., 1024 .. and 7936 ..)
        spoil(sx, torch.tensor([300, 1024, 7950], device="cuda"))
    if scales == "some features":
        spoil(sw, torch.tensor([0, 777, 2 * hidden - 1], device="cuda"))
    kw = dict(activation=act, accum=FAST)
    f32 = te.te_fp8_gated_fwd(x, sx, E4, w, sw, E4, out_dtype=F32, need_z=True, **kw)
    z, ez, y, bound = forward64(x, sx, E4, w, sw, E4, act, False)
    close(f32.z, z, ez + 2.0 ** -8 * (z.abs() + ez), "z")
    close(f32.y, y, bound + U * y.abs(), "y")
    del z, ez, y, bound
    assert (f32.y != 0).any()
    assert torch.equal(te.te_fp8_gated_fwd(x, sx, E4, w, sw, E4, out_dtype=BF, **kw).y, f32.y.bfloat16())
    for rowwise, transpose in ((True, False), (False, True), (True, True)):
        if transpose and rows % 128:
            continue
        r = te.te_fp8_gated_fwd(x, sx, E4, w, sw, E4, out_dtype=E4, flags=te.TE_CAST_POW2_SCALE, rowwise=rowwise, transpose=transpose,
                                need_z=True, **kw)
        assert torch.equal(r.z, f32.z)
        check_casts(r, f32.y, hidden, rows, E4, True)
    again = te.te_fp8_gated_fwd(x, sx, E4, w, sw, E4, out_dtype=F32, need_z=True, **kw)
    assert torch.equal(again.y, f32.y) and torch.equal(again.z, f32.z)
    # other formats take FULL's update (read as e5m2, some of x's codes are infinite or NaN)
    full = te.te_fp8_gated_fwd(x, sx, E5, w, sw, E4, out_dtype=F32, activation=act)
    fast = te.te_fp8_gated_fwd(x, sx, E5, w, sw, E4, out_dtype=F32, **kw)
    assert torch.allclose(fast.y, full.y, rtol=0.0, atol=0.0, equal_nan=True)


@pytest.mark.parametrize("rows", [256, 512])
def test_parts_and_tiles_on_power_of_two_scales(rows):
    """Where every scale is a power of two, parts of 64 x 128 and tiles of 256 x 256 chain the same blocks in the same order, so
    the outputs that are asked for change nothing; where some are not, either is within the bound of the products."""
    k, hidden = 1152, 640
    g = gen(rows)
    x, sx = operand(g, rows, k, E4, pow2=True)
    w, sw = operand(g, 2 * hidden, k, E4, 1.5 * k ** -0.5, pow2=True)

    def outputs():
        return [te.te_fp8_gated_fwd(x, sx, E4, w, sw, E4, need_z=True, accum=FAST, **kw)
                for kw in (dict(out_dtype=F32), dict(out_dtype=E4), dict(out_dtype=E4, transpose=True), dict(out_dtype=E4, rowwise=False, transpose=True))]

    plain, *casts = outputs()
    for c in casts:
        assert torch.equal(c.z, plain.z)
        check_casts(c, plain.y, hidden, rows, E4)
    spoil(sx, torch.tensor([70], device="cuda"))
    z, ez, y, bound = forward64(x, sx, E4, w, sw, E4, SILU, False)
    for r in outputs():
        close(r.z, z, ez + 2.0 ** -8 * (z.abs() + ez), "z")
        if r.y is not None:
            close(r.y, y, bound + U * y.abs(), "y")


@pytest.mark.parametrize("rows", [1, 16, 77, 128, 129, 256, 384, 600])
@pytest.mark.parametrize("k", [128, 1024])
@pytest.mark.parametrize("out,pow2", [(E4, False), (E5, True)])
def test_one_group_of_features(rows, k, out, pow2):
    """Hidden size 128: one fp8 group to a row of y, two to a row of dz."""
    hidden = 128
    g = gen(rows + k)
    x, sx = operand(g, rows, k, E4)
    w, sw = operand(g, 2 * hidden, k, E4, 1.5 * k ** -0.5)
    wt, swt = operand(g, hidden, k, E4, k ** -0.5)
    dy, sdy = operand(g, rows, k, E5, 1e-2)
    flags = te.TE_CAST_POW2_SCALE if pow2 else 0
    plain = te.te_fp8_gated_fwd(x, sx, E4, w, sw, E4, out_dtype=F32, need_z=True)
    z, ez, y, bound = forward64(x, sx, E4, w, sw, E4, SILU, rows <= 128)
    close(plain.y, y, bound + U * y.abs(), "y")
    grad = te.te_fp8_gated_dgrad(dy, sdy, E5, wt, swt, E4, plain.z, out_dtype=F32)
    dz, e = dgrad64(dy, sdy, E5, wt, swt, E4, plain.z, SILU)
    close(grad.dz, dz, e + U * dz.abs(), "dz")
    assert (plain.y != 0).all(1).any() and (grad.dz != 0).all(1).any()
    for rowwise, transpose in ((True, False), (False, True), (True, True)):
        if transpose and rows % 128:
            continue
        kw = dict(out_dtype=out, flags=flags, rowwise=rowwise, transpose=transpose)
        check_casts(te.te_fp8_gated_fwd(x, sx, E4, w, sw, E4, **kw), plain.y, hidden, rows, out, pow2)
        check_casts(te.te_fp8_gated_dgrad(dy, sdy, E5, wt, swt, E4, plain.z, **kw), grad.dz, 2 * hidden, rows, out, pow2)
