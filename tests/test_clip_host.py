"""Host side of te_grad_norm_clip over long lists of tensors (CPU only)."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
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


class Launch(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("which", "first_count", "tensors", "chunks", "slots", "past", "norm")]


@pytest.fixture(scope="module")
def recorder(tmp_path_factory):
    """The front end with launchers that only note their arguments."""
    if shutil.which("g++") is None:
        pytest.skip("no host compiler")
    out = str(tmp_path_factory.mktemp("clip") / "libte_fp8_record.so")
    csrc, sub = os.path.join(ROOT, "fp8_linear_layer_amd", "csrc"), os.path.join(ROOT, "tests", "sanitize")
    subprocess.run(["g++", "-std=c++17", "-fPIC", "-shared", "-O1", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    "-I", os.path.join(ROOT, "include"), "-I", csrc, os.path.join(csrc, "api.cpp"), os.path.join(csrc, "api_ops.cpp"),
                    os.path.join(sub, "host_stubs.cpp"), os.path.join(sub, "host_record_clip.cpp"), "-o", out], check=True)
    lib = ctypes.CDLL(out)
    lib.recorded.restype = ctypes.c_int64
    lib.te_grad_norm_clip.argtypes = [ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                      ctypes.c_void_p]

    def launches(counts, dtype=te.TE_DTYPE_F32):
        arr = (ops._GradTensor * max(1, len(counts)))(*[(0x10000, 0x20000, n, dtype, te.TE_DTYPE_F32) for n in counts])
        assert lib.te_grad_norm_clip(arr, len(counts), 1.0, 0x30000, 0x40000, 1 << 20, None) == 0
        got = (Launch * 2000)()
        return list(got[:lib.recorded(got, 2000)])
    return launches


def split(launches):
    return [x for x in launches if x.which == 0], [x for x in launches if x.which == 1]


@pytest.mark.parametrize("counts", [[], [0], [5], [100] * 96, [100] * 97, [100 + i for i in range(1000)], [10 ** 7] * 200, [0] * 200])
def test_every_tensor_is_in_one_launch_of_each_pass(recorder, counts):
    sums, scales = split(recorder(counts))
    live = [n for n in counts if n]
    for launches in (sums, scales):
        assert sum(x.tensors for x in launches) == len(live) and sum(x.chunks for x in launches) == sum(-(-n // 8192) for n in live)
    assert [x.norm for x in scales].count(1) == 1
    blocks = [min(1024, max(1, x.chunks)) for x in sums]
    assert [x.slots for x in sums] == [max(blocks[:i], default=0) for i in range(len(blocks))]
    assert all(x.slots == max(blocks) for x in scales)


def test_past_the_caches_goes_by_the_whole_list(recorder):
    """Gradients of a gigabyte are far larger than the caches, in whatever number of tensors they come."""
    mebi = 1 << 20
    for counts in ([300 * mebi], [mebi] * 300, [mebi // 16] * 4800):
        assert all(x.past for x in recorder(counts))
        assert all(x.past for x in recorder(counts, te.TE_DTYPE_BF16))
    for counts in ([16 * mebi], [mebi] * 16, [mebi // 16] * 256, [100] * 50000):
        assert not any(x.past for x in recorder(counts))
    assert all(x.past for x in recorder([150 * mebi])) and not any(x.past for x in recorder([150 * mebi], te.TE_DTYPE_BF16))


def test_second_pass_starts_where_the_first_ended(recorder):
    """Last launch first: what the first pass read last is what the caches still hold."""
    sums, scales = split(recorder([1000 + i for i in range(500)]))
    assert [x.first_count for x in scales] == [x.first_count for x in reversed(sums)]
    assert len(sums) == 6


def test_an_empty_lists_norm_belongs_to_the_given_stream(monkeypatch):
    """Without gradients the norm is allocated here: for the stream that writes it, like every other output."""
    current, seen = ["default"], []

    class Stream:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            self.before, current[0] = current[0], self.s or current[0]

        def __exit__(self, *_):
            current[0] = self.before

    class Native:
        @staticmethod
        def grad_norm_clip(grads, max_norm, out, norm, workspace):
            seen.append(("call", current[0]))
            return norm

    empty = torch.empty
    monkeypatch.setattr(torch.cuda, "stream", Stream)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: seen.append(("empty", current[0])) or empty(1))
    monkeypatch.setattr(ops, "_native", Native)
    te.te_grad_norm_clip([], 1.0, stream="side")
    te.te_grad_norm_clip([], 1.0)
    assert seen == [("empty", "side"), ("call", "side"), ("empty", "default"), ("call", "default")]
