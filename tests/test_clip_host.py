"""Host side of te_grad_norm_clip over long lists of tensors (CPU only)."""
import os

import pytest

te = pytest.importorskip("fp8_linear_layer_amd")
from fp8_linear_layer_amd import ops  # noqa: E402


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(te.LIB_PATH):
        pytest.skip("libte_fp8.so not built")
    return ops._lib()


def test_partial_sums_do_not_grow_with_the_list(lib):
    """Every workgroup of every launch of the second pass adds all partial sums up: with a list of them per launch
    that work grew with the square of the tensors."""
    sizes = {n: lib.te_grad_norm_workspace_bytes(n) for n in (0, 1, 96, 97, 1000, 18000, 1 << 20)}
    assert len(set(sizes.values())) == 1 and 0 < sizes[1] <= 8192, sizes
