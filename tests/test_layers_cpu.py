"""Host-side refusals of the layer operators' C entry points (no kernel is
launched: fake device addresses fail validation first), and the same checks
under a host-only ASan/UBSan build of api_layers.cpp."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = [0x100000000 * (i + 1) for i in range(16)]
OK, NULL, SHAPE, LD, ALIGN, UNSUP, DEVICE, LAUNCH, ALIAS = range(9)


@pytest.fixture(scope="module")
def lib():
    import torch
    from fine_grained_fp8_amd import _lib, build
    if torch.cuda.is_available():
        pytest.skip("valid calls on made-up addresses: only where no GPU can run them")
    sanitized = os.environ.get("FP8BS_SANITIZED_LAYERS")
    if sanitized:
        return _lib.load_library(sanitized)
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.load_library()


def call(f, order, base, **change):
    assert set(change) <= set(order), change
    return f(*[{**base, **change}[k] for k in order])


NORM = "x rows cols ldx xt w b wt eps y ldy mean rstd q ldq s ld_s stream".split()


def norm(lib, **c):
    base = dict(x=P[0], rows=64, cols=256, ldx=256, xt=0, w=P[1], b=P[2], wt=1, eps=1e-5, y=P[3], ldy=256, mean=P[4],
                rstd=P[5], q=P[6], ldq=256, s=P[7], ld_s=64, stream=None)
    return call(lib.fp8_layer_norm, NORM, base, **c)


def test_layer_norm_validation(lib):
    assert norm(lib) in (DEVICE, OK)
    assert norm(lib, xt=2) == UNSUP and norm(lib, wt=-1) == UNSUP
    assert norm(lib, rows=-1) == SHAPE and norm(lib, cols=200) == SHAPE and norm(lib, eps=-1.0) == SHAPE
    assert norm(lib, eps=float("nan")) == SHAPE
    assert norm(lib, cols=16384 + 128, ldx=20000, ldy=20000, ldq=20000) == UNSUP
    assert norm(lib, rows=0, x=None) == OK and norm(lib, cols=0, x=None) == OK
    assert norm(lib, x=None) == NULL and norm(lib, s=None) == NULL and norm(lib, q=None) == NULL
    assert norm(lib, y=None, q=None, s=None) == NULL
    assert norm(lib, y=None) in (DEVICE, OK) and norm(lib, q=None, s=None) in (DEVICE, OK)
    for k in ("ldx", "ldy", "ldq"):
        assert norm(lib, **{k: 255}) == LD
        assert norm(lib, **{k: 1 << 60}) == UNSUP
    assert norm(lib, ld_s=63) == LD
    assert norm(lib, x=P[0] + 2) == ALIGN and norm(lib, w=P[1] + 4) == ALIGN and norm(lib, ldx=257) == ALIGN
    plain = dict(q=None, s=None)
    assert norm(lib, x=P[0] + 2, ldx=257, w=P[1] + 4, **plain) in (DEVICE, OK)
    assert norm(lib, x=P[0] + 1, **plain) == ALIGN and norm(lib, mean=P[4] + 2, **plain) == ALIGN
    for k, v in (("y", P[0]), ("q", P[0] + 256), ("s", P[1]), ("mean", P[3] + 512), ("rstd", P[4] + 4), ("q", P[7])):
        assert norm(lib, **{k: v}) == ALIAS, k


GRAD = "dy lddy x ldx rows cols xt mean rstd w wt dx lddx dw db ws bytes stream".split()


def grad(lib, **c):
    base = dict(dy=P[0], lddy=250, x=P[1], ldx=250, rows=64, cols=250, xt=1, mean=P[2], rstd=P[3], w=P[4], wt=0, dx=P[5],
                lddx=250, dw=P[6], db=P[7], ws=P[8], bytes=lib.fp8_layer_norm_backward_workspace(64, 250), stream=None)
    return call(lib.fp8_layer_norm_backward, GRAD, base, **c)


def test_layer_norm_backward_validation(lib):
    assert lib.fp8_layer_norm_backward_workspace(64, 250) > 0
    assert lib.fp8_layer_norm_backward_workspace(0, 250) == 0
    assert lib.fp8_layer_norm_backward_workspace(-1, 250) == -1
    assert lib.fp8_layer_norm_backward_workspace(64, 16385) == -1
    assert grad(lib) in (DEVICE, OK)
    assert grad(lib, dw=None, db=None) in (DEVICE, OK) and grad(lib, w=None) in (DEVICE, OK)
    assert grad(lib, rows=0, dw=None, db=None) == OK and grad(lib, cols=0) == OK
    for k in ("dy", "x", "mean", "rstd", "dx", "ws"):
        assert grad(lib, **{k: None}) == NULL, k
    assert grad(lib, bytes=16) == SHAPE and grad(lib, rows=-1) == SHAPE
    for k in ("lddy", "ldx", "lddx"):
        assert grad(lib, **{k: 249}) == LD
    assert grad(lib, xt=7) == UNSUP and grad(lib, cols=20000) == UNSUP
    assert grad(lib, x=P[1] + 2) == ALIGN and grad(lib, ws=P[8] + 4) == ALIGN
    for k, v in (("dx", P[0]), ("dx", P[1] + 4), ("dw", P[5]), ("db", P[6] + 4), ("ws", P[2]), ("dw", P[8])):
        assert grad(lib, **{k: v}) == ALIAS, k


MOE = ("T H I E first local k x ldx router ld_r bias gate norm scale w13 s13 w2 s2 y yt ldy ids gates ws bytes "
       "stream").split()


def moe(lib, **c):
    base = dict(T=8, H=256, I=384, E=16, first=4, local=4, k=2, x=P[0], ldx=256, router=P[1], ld_r=256, bias=None, gate=0,
                norm=1, scale=1.0, w13=P[2], s13=P[3], w2=P[4], s2=P[5], y=P[6], yt=0, ldy=256, ids=P[7], gates=P[8],
                ws=P[9], bytes=lib.fp8_moe_few_tokens_workspace(8, 256, 384, 16, 4, 2), stream=None)
    return call(lib.fp8_moe_few_tokens, MOE, base, **c)


def test_moe_validation(lib):
    f = lib.fp8_moe_few_tokens_workspace
    assert f(8, 256, 384, 16, 4, 2) > 0 and f(65, 256, 384, 16, 4, 2) == -1 and f(8, 200, 384, 16, 4, 2) == -1
    assert moe(lib) in (DEVICE, OK) and moe(lib, ids=None, gates=None) in (DEVICE, OK)
    assert moe(lib, gate=1, bias=P[10]) in (DEVICE, OK) and moe(lib, bias=P[10]) == UNSUP
    assert moe(lib, T=0, x=None) == OK
    assert moe(lib, T=65) == UNSUP and moe(lib, k=17, E=32) == UNSUP and moe(lib, E=1025) == UNSUP and moe(lib, gate=2) == UNSUP
    for c in (dict(T=-1), dict(H=200), dict(I=100), dict(k=0), dict(k=17), dict(first=13), dict(first=-1), dict(local=0),
              dict(E=0), dict(bytes=256)):
        assert moe(lib, **c) == SHAPE, c
    for k in ("x", "router", "w13", "s13", "w2", "s2", "y", "ws"):
        assert moe(lib, **{k: None}) == NULL, k
    for k in ("ldx", "ld_r", "ldy"):
        assert moe(lib, **{k: 248}) == LD
        assert moe(lib, **{k: 260}) == ALIGN
    for k in ("x", "router", "w13", "w2", "y", "ws"):
        assert moe(lib, **{k: P[11] + 8}) == ALIGN, k
    for k, v in (("y", P[0]), ("ids", P[1]), ("gates", P[7]), ("ws", P[2] + 4096), ("y", P[9])):
        assert moe(lib, **{k: v}) == ALIAS, k


ADAPTER = "T N K r n x ldx W sW ld_sw A B ids scales C ct ldc ws bytes stream".split()


def adapter(lib, **c):
    base = dict(T=8, N=384, K=256, r=16, n=3, x=P[0], ldx=256, W=P[1], sW=P[2], ld_sw=2, A=P[3], B=P[4], ids=P[5], scales=P[6],
                C=P[7], ct=0, ldc=384, ws=P[8], bytes=lib.fp8_adapter_linear_workspace(c.get("T", 8), 384, 256, 16, 3),
                stream=None)
    return call(lib.fp8_adapter_linear, ADAPTER, base, **c)


def test_adapter_validation(lib):
    f = lib.fp8_adapter_linear_workspace
    assert f(8, 384, 256, 16, 3) > 0 and f(8, 384, 256, 12, 3) == -1 and f(8, 384, 256, 136, 3) == -1
    for T in (8, 4096):
        assert adapter(lib, T=T) in (DEVICE, OK)
        assert adapter(lib, T=T, scales=None) in (DEVICE, OK)
        assert adapter(lib, T=T, bytes=1024) == SHAPE
    assert adapter(lib, T=0, x=None) == OK
    for c in (dict(T=-1), dict(N=200), dict(K=200), dict(r=0), dict(r=12), dict(n=0)):
        assert adapter(lib, **{**c, "bytes": 1 << 30}) == SHAPE, c
    assert adapter(lib, r=136) == UNSUP and adapter(lib, ct=3) == UNSUP
    for k in ("x", "W", "sW", "A", "B", "ids", "C", "ws"):
        assert adapter(lib, **{k: None}) == NULL, k
    assert adapter(lib, ldx=248) == LD and adapter(lib, ldc=376) == LD and adapter(lib, ld_sw=1) == LD
    assert adapter(lib, ldx=260) == ALIGN and adapter(lib, ldc=388) == ALIGN
    for k in ("x", "W", "A", "B", "C", "ws"):
        assert adapter(lib, **{k: P[9] + 8}) == ALIGN, k
    for k, v in (("C", P[0]), ("C", P[5]), ("ws", P[1]), ("ws", P[7])):
        assert adapter(lib, **{k: v}) == ALIAS, k


def test_layer_validation_under_asan_ubsan(tmp_path):
    """api_layers.cpp built on the host with sanitizers, its launchers
    replaced by stubs, runs the validation tests above without a report."""
    if os.environ.get("FP8BS_SANITIZED_LAYERS"):
        pytest.skip("already the sanitized child run")
    gxx = shutil.which("g++")
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    if not gxx or not os.path.exists(os.path.join(rocm, "include", "hip", "hip_runtime.h")):
        pytest.skip("g++ or the HIP headers are not available")
    so = str(tmp_path / "liblayers_san.so")
    csrc = os.path.join(ROOT, "fine_grained_fp8_amd", "csrc")
    r = subprocess.run([gxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined",
                        "-fno-omit-frame-pointer", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__",
                        "-I", os.path.join(rocm, "include"), "-I", os.path.join(ROOT, "include"), "-I", csrc,
                        os.path.join(csrc, "api_layers.cpp"), os.path.join(ROOT, "tests", "c", "layer_stubs.cpp"),
                        "-L", os.path.join(rocm, "lib"), "-Wl,-rpath," + os.path.join(rocm, "lib"), "-lamdhip64", "-o", so],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    asan = subprocess.run([gxx, "-print-file-name=libasan.so"], capture_output=True, text=True).stdout.strip()
    env = dict(os.environ, LD_PRELOAD=asan, FP8BS_SANITIZED_LAYERS=so, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([sys.executable, "-m", "pytest", os.path.abspath(__file__), "-q", "-x", "-p", "no:cacheprovider",
                        "-k", "validation and not asan"], env=env, capture_output=True, text=True, timeout=600, cwd=ROOT)
    report = r.stdout[-3000:] + r.stderr[-3000:]
    assert r.returncode == 0 and " passed" in r.stdout, report
    assert "AddressSanitizer" not in r.stderr and "runtime error" not in r.stderr, report
