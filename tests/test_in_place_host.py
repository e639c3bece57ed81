"""Sums in place (CPU only): an output that is an input's own buffer at another row stride would have rows written over
rows that are still to be read, so the C ABI refuses it before anything is enqueued.  Pointers are dummies."""
import os

import pytest

te = pytest.importorskip("fp8_linear_layer_amd")
from fp8_linear_layer_amd import block_ops, ops  # noqa: E402

BF, F32 = te.TE_DTYPE_BF16, te.TE_DTYPE_F32
INV = 1
A, B, C, D, S, T, W, G = (0x10000 * i for i in range(1, 9))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(te.LIB_PATH):
        pytest.skip("libte_fp8.so not built")
    ops._lib()
    return block_ops._lib()


def refused(lib, status):
    assert status == INV
    assert "in place" in lib.te_last_error_message().decode()


@pytest.mark.parametrize("ld_res,ld_h", [(256, 264), (264, 256), (512, 256)])
@pytest.mark.parametrize("rows", [2, 128])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_layernorm_fwd(lib, rows, ld_res, ld_h, dtype):
    refused(lib, lib.te_layernorm_fwd(A, BF, 256, S, dtype, ld_res, 0.0, None, B, T, 1e-5, rows, 256, S, ld_h, C, G, D, BF, 256, 0, None,
                                      None, 0, None, None))


@pytest.mark.parametrize("ld_res,ld_dh", [(256, 264), (264, 256), (512, 256)])
@pytest.mark.parametrize("rows", [2, 128])
@pytest.mark.parametrize("p", [0.0, 0.5])
def test_layernorm_bwd(lib, rows, ld_res, ld_dh, p):
    drop = (p, G, T, BF, 256) if p else (0.0, None, None, BF, 0)
    refused(lib, lib.te_layernorm_bwd(A, BF, 256, B, BF, 256, C, C, D, rows, 256, S, ld_res, S, ld_dh, *drop, None, None, None, 0, None))


@pytest.mark.parametrize("ld_res,ld_h", [(256, 264), (264, 256), (512, 256)])
@pytest.mark.parametrize("rows", [2, 128])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rmsnorm_fwd(lib, rows, ld_res, ld_h, dtype):
    refused(lib, lib.te_rmsnorm_fwd(A, BF, 256, S, dtype, ld_res, B, 1e-5, rows, 256, S, ld_h, C, D, BF, 256, 0, None, None, 0, None, None))


@pytest.mark.parametrize("ld_res,ld_dh", [(256, 264), (264, 256), (512, 256)])
@pytest.mark.parametrize("rows", [2, 128])
def test_rmsnorm_bwd(lib, rows, ld_res, ld_dh):
    refused(lib, lib.te_rmsnorm_bwd(A, BF, 256, B, BF, 256, C, D, rows, 256, S, ld_res, S, ld_dh, None, None, 0, None))
