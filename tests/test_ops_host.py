"""Host-side checks of the operators' C ABI (include/te_ops.h) and of their Python binding (CPU only).

Each rejected C call returns its status before anything is enqueued; its pointers are dummies that
are never dereferenced.  The binding refuses tensors whose pointers must not reach a kernel."""
import ctypes
import math
import os
import re
import shutil
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
te = pytest.importorskip("fp8_linear_layer_amd")
from fp8_linear_layer_amd import ops  # noqa: E402

E4, E5, BF, F32 = te.TE_DTYPE_E4M3, te.TE_DTYPE_E5M2, te.TE_DTYPE_BF16, te.TE_DTYPE_F32
INV, MISAL, UNSUP = 1, 2, 3
A, B, C, D, S, T = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000, 0x60000


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(te.LIB_PATH):
        pytest.skip("libte_fp8.so not built")
    return ops._lib()


def test_every_declared_function_is_exported_and_bound(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "te_ops.h")).read(), flags=re.S)
    declared = set(re.findall(r"\b(te_[a-z0-9_]+)\s*\(", text))
    assert declared == set(ops.EXPORTED)
    assert all(getattr(lib, f).argtypes is not None for f in declared)


def refused(lib, status, want):
    assert status == want
    assert lib.te_last_error_message().decode()


def norm_fwd(lib, x=A, xd=BF, ldx=256, res=None, rd=0, ldr=0, gamma=B, eps=1e-5, rows=128, cols=256, h=None, ldh=0, rstd=C, y=D,
             yd=BF, ldy=256, flags=0, s=None, qt=None, ldqt=0, st=None):
    return lib.te_rmsnorm_fwd(x, xd, ldx, res, rd, ldr, gamma, eps, rows, cols, h, ldh, rstd, y, yd, ldy, flags, s, qt, ldqt, st, None)


Q = dict(yd=E4, s=S)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INV), (dict(gamma=None), INV), (dict(rstd=None), INV), (dict(y=None), INV),
    (dict(rows=-1), INV), (dict(rows=1 << 31), INV), (dict(cols=0), INV), (dict(cols=-5), INV), (dict(cols=32769, ldx=40000, ldy=40000), UNSUP),
    (dict(xd=E4), INV), (dict(xd=0), INV), (dict(yd=0), INV), (dict(yd=7), INV),
    (dict(ldx=255), INV), (dict(ldy=255), INV),
    (dict(eps=-1.0), INV), (dict(eps=math.nan), INV), (dict(eps=math.inf), INV),
    (dict(x=A + 1), MISAL), (dict(xd=F32, x=A + 2), MISAL), (dict(gamma=B + 1), MISAL), (dict(rstd=C + 2), MISAL), (dict(y=D + 1), MISAL),
    (dict(h=T, ldh=256), INV),                                        # h without a residual
    (dict(res=S, rd=BF, ldr=256), INV),                               # a residual without h
    (dict(res=S, rd=BF, ldr=255, h=T, ldh=256), INV), (dict(res=S, rd=BF, ldr=256, h=T, ldh=200), INV),
    (dict(res=S, rd=E5, ldr=256, h=T, ldh=256), INV), (dict(res=S, rd=F32, ldr=256, h=T + 2, ldh=256), MISAL),
    (dict(flags=1), INV), (dict(s=S), INV), (dict(qt=T, ldqt=128, st=S), INV),     # fp8's own arguments on a bf16 output
    (dict(yd=E4), INV), (dict(yd=E4, s=S, flags=2), INV), (dict(yd=E4, y=None), INV),
    (dict(cols=200, **Q), INV), (dict(ldy=264, **Q), MISAL), (dict(y=D + 8, **Q), MISAL), (dict(yd=E4, s=S + 4), MISAL),
    (dict(qt=T, ldqt=128, **Q), INV), (dict(st=T, **Q), INV), (dict(qt=T, ldqt=112, st=T, **Q), INV),
    (dict(qt=T, ldqt=136, st=T, **Q), MISAL), (dict(qt=T + 8, ldqt=128, st=T, **Q), MISAL),
    (dict(rows=100, qt=T, ldqt=128, st=T, **Q), INV), (dict(yd=E4, y=None, cols=252, ldx=256, qt=T, ldqt=128, st=T), INV),
    (dict(x=A + 2, qt=T, ldqt=128, st=T, **Q), MISAL), (dict(ldx=260, qt=T, ldqt=128, st=T, **Q), MISAL),
])
def test_norm_forward_rejects(lib, kw, status):
    refused(lib, norm_fwd(lib, **kw), status)


def norm_bwd(lib, dy=A, yd=BF, ldy=256, h=B, hd=BF, ldh=256, rstd=C, gamma=D, rows=64, cols=256, dres=None, ldr=0, dh=S, lddh=256,
             dg=T, ws=0x70000, wsb=1 << 30):
    return lib.te_rmsnorm_bwd(dy, yd, ldy, h, hd, ldh, rstd, gamma, rows, cols, dres, ldr, dh, lddh, dg, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), INV), (dict(h=None), INV), (dict(rstd=None), INV), (dict(gamma=None), INV), (dict(dh=None), INV),
    (dict(rows=-2), INV), (dict(cols=0), INV), (dict(cols=1 << 16, ldy=1 << 16, ldh=1 << 16, lddh=1 << 16), UNSUP),
    (dict(yd=E4), INV), (dict(hd=E5), INV), (dict(ldy=100), INV), (dict(ldh=255), INV), (dict(lddh=255), INV),
    (dict(dres=A, ldr=255), INV), (dict(dres=A + 1, ldr=256), MISAL), (dict(dg=T + 2), MISAL), (dict(dy=A + 1), MISAL),
    (dict(ws=None), INV), (dict(wsb=64), INV), (dict(ws=0x70008), MISAL),
])
def test_norm_backward_rejects(lib, kw, status):
    refused(lib, norm_bwd(lib, **kw), status)


def router_fwd(lib, v=A, vd=BF, ld=64, tokens=100000, experts=64, k=6, renorm=0, mask=None, index=B, weight=C, lse=D, counts=S, routed=T,
               loss=T + 16, ws=0x70000, wsb=1 << 30):
    return lib.te_moe_router_fwd(v, vd, ld, tokens, experts, k, renorm, mask, index, weight, lse, counts, routed, loss, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(v=None), INV), (dict(index=None), INV), (dict(weight=None), INV), (dict(vd=E4), INV), (dict(vd=0), INV),
    (dict(ld=63), INV), (dict(tokens=-1), INV), (dict(tokens=1 << 31), INV), (dict(experts=0), INV), (dict(k=0), INV), (dict(k=65), INV),
    (dict(k=17), UNSUP), (dict(experts=2049, ld=2049), UNSUP),
    (dict(counts=None), INV), (dict(routed=None), INV), (dict(loss=None), INV),
    (dict(ws=None), INV), (dict(wsb=16), INV), (dict(ws=0x70004), MISAL),
    (dict(v=A + 1), MISAL), (dict(vd=F32, v=A + 2), MISAL), (dict(index=B + 2), MISAL), (dict(lse=D + 1), MISAL), (dict(loss=T + 18), MISAL),
])
def test_router_forward_rejects(lib, kw, status):
    refused(lib, router_fwd(lib, **kw), status)


def router_bwd(lib, v=A, vd=F32, ld=64, tokens=10, experts=64, k=6, index=B, lse=C, dw=D, counts=S, routed=S + 512, dl=T, d=0x70000, ldd=64):
    return lib.te_moe_router_bwd(v, vd, ld, tokens, experts, k, 0, index, lse, dw, counts, routed, dl, d, ldd, None)


@pytest.mark.parametrize("kw,status", [
    (dict(v=None), INV), (dict(index=None), INV), (dict(lse=None), INV), (dict(d=None), INV), (dict(vd=E5), INV),
    (dict(ld=63), INV), (dict(ldd=63), INV), (dict(tokens=-1), INV), (dict(experts=0), INV), (dict(k=65), INV), (dict(k=20), UNSUP),
    (dict(counts=None), INV), (dict(routed=None), INV), (dict(dw=D + 2), MISAL), (dict(dl=T + 1), MISAL), (dict(d=0x70002), MISAL),
])
def test_router_backward_rejects(lib, kw, status):
    refused(lib, router_bwd(lib, **kw), status)


def clip(lib, tensors=((A, B, 100, F32, BF),), n=None, max_norm=1.0, norm=C, ws=D, wsb=1 << 20):
    arr = (ops._GradTensor * max(len(tensors), 1))(*tensors) if tensors is not None else None
    return lib.te_grad_norm_clip(arr, len(tensors) if n is None else n, max_norm, norm, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(tensors=None, n=1), INV), (dict(n=-1), INV), (dict(norm=None), INV), (dict(norm=C + 2), MISAL),
    (dict(max_norm=0.0), INV), (dict(max_norm=-1.0), INV), (dict(max_norm=math.nan), INV),
    (dict(ws=None), INV), (dict(wsb=100), INV), (dict(ws=D + 8), MISAL),
    (dict(tensors=((None, B, 5, F32, F32),)), INV), (dict(tensors=((A, B, -1, F32, F32),)), INV),
    (dict(tensors=((A, B, 5, E4, F32),)), INV), (dict(tensors=((A, B, 5, F32, 0),)), INV),
    (dict(tensors=((A, B, 5, BF, BF), (A + 1, B, 5, BF, BF))), MISAL), (dict(tensors=((A, B + 2, 5, F32, F32),)), MISAL),
    (dict(tensors=((A, A, 5, F32, BF),)), INV), (dict(tensors=((A, B, (1 << 36) + 1, F32, F32),)), UNSUP),
])
def test_clip_rejects(lib, kw, status):
    refused(lib, clip(lib, **kw), status)


def test_empty_calls_need_no_pointers(lib):
    assert norm_fwd(lib, x=None, gamma=None, rstd=None, y=None, rows=0) == 0
    assert router_fwd(lib, v=None, index=None, weight=None, lse=None, counts=None, routed=None, loss=None, tokens=0) == 0
    assert router_bwd(lib, v=None, index=None, lse=None, d=None, tokens=0) == 0
    assert lib.te_last_error_message().decode() == ""


def test_workspace_sizes(lib):
    assert lib.te_rmsnorm_bwd_workspace_bytes(0, 100) == 0 and lib.te_rmsnorm_bwd_workspace_bytes(1, 5) >= 32
    assert lib.te_moe_router_workspace_bytes(0, 8) == 0 and lib.te_moe_router_workspace_bytes(1, 8) == 0
    big = [lib.te_moe_router_workspace_bytes(1 << 30, e) for e in (8, 64, 256, 2048)]
    assert all(b > 0 for b in big) and big[-1] < 1 << 26
    assert lib.te_grad_norm_workspace_bytes(0) > 0 and lib.te_grad_norm_workspace_bytes(-1) == 0
    assert lib.te_grad_norm_workspace_bytes(10000) < 1 << 21


CPU = torch.zeros((4, 128), dtype=torch.bfloat16)


@pytest.mark.parametrize("call", [
    lambda: te.te_rmsnorm_fwd(CPU, CPU[0]),
    lambda: te.te_rmsnorm_fwd(CPU[0], CPU[0]),
    lambda: te.te_rmsnorm_bwd(CPU, CPU, CPU.float()[:, 0], CPU[0]),
    lambda: te.te_moe_router_fwd(CPU, 2),
    lambda: te.te_moe_router_bwd(CPU, torch.zeros((4, 2), dtype=torch.int32), torch.zeros(4)),
    lambda: te.te_grad_norm_clip([CPU], 1.0),
])
def test_binding_refuses_tensors_off_the_gpu(lib, call):
    with pytest.raises(te.TeFp8Error, match="GPU|expected a tensor"):
        call()


SAN = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer", "-g", "-O1"]


@pytest.mark.skipif(shutil.which("g++") is None or "TE_FP8_TEST_LIB" in os.environ, reason="no host compiler, or already under it")
def test_validation_under_sanitizers(tmp_path):
    """The two front ends with stand-ins for the kernels (every launch reports an error), instrumented,
    run the tests above in a child process."""
    out = str(tmp_path / "libte_fp8_host_san.so")
    csrc = os.path.join(ROOT, "fp8_linear_layer_amd", "csrc")
    sub = os.path.join(ROOT, "tests", "sanitize")
    subprocess.run(["g++", "-std=c++17", "-fPIC", "-shared", *SAN, "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    "-I", os.path.join(ROOT, "include"), "-I", csrc, os.path.join(csrc, "api.cpp"), os.path.join(csrc, "api_ops.cpp"),
                    os.path.join(sub, "host_stubs.cpp"), os.path.join(sub, "host_stubs_ops.cpp"), "-o", out], check=True)
    # (the C++ runtime beside the sanitizer's: the binding throws, and the sanitizer wants to know how before that)
    preload = [subprocess.check_output(["gcc", f"-print-file-name={n}"], text=True).strip() for n in ("libasan.so", "libstdc++.so.6")]
    env = dict(os.environ, LD_PRELOAD=" ".join(preload), TE_FP8_TEST_LIB=out, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-m", "not gpu",
                        os.path.abspath(__file__)], cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    text = r.stdout + r.stderr
    assert "AddressSanitizer" not in text and "runtime error:" not in text, text[-4000:]
    assert r.returncode == 0 and " passed" in r.stdout, text[-4000:]
