"""Host-side refusals of the C entry points of api_blocks.cpp (no kernel is
launched: fake device addresses fail validation first), and the same checks
under a host-only ASan/UBSan build of that file."""
import ctypes
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = [0x1000000000 * (i + 1) for i in range(24)]
OK, NULL, SHAPE, LD, ALIGN, UNSUP, DEVICE, LAUNCH, ALIAS = range(9)
PASSED = (DEVICE, OK)      # everything up to the device


@pytest.fixture(scope="module")
def lib():
    import torch
    from fine_grained_fp8_amd import _lib, build
    if torch.cuda.is_available():
        pytest.skip("valid calls on made-up addresses: only where no GPU can run them")
    sanitized = os.environ.get("FP8BS_SANITIZED_BLOCKS")
    if sanitized:
        return _lib.load_library(sanitized)
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.load_library()


def call(f, order, base, change):
    assert set(change) <= set(order), change
    return f(*[{**base, **change}[k] for k in order])


GATED = "M I K A lda sA ld_sa W s13 ld_s13 act h ht ldh gu ld_gu q ldq s ld_s ws bytes stream".split()


def gated(lib, **c):
    base = dict(M=8, I=256, K=384, A=P[0], lda=384, sA=P[1], ld_sa=8, W=P[2], s13=P[3], ld_s13=3, act=0, h=P[4], ht=0, ldh=256,
                gu=P[5], ld_gu=512, q=None, ldq=256, s=None, ld_s=8, ws=P[8], bytes=1 << 24, stream=None)
    return call(lib.fp8_block_gemm_gated, GATED, base, c)


@pytest.mark.parametrize("M", [8, 200, 16384])
def test_gated_validation(lib, M):
    def g(**c):
        return gated(lib, **{"M": M, "ld_sa": M, "ld_s": M, "ws": P[9], **c})
    f = lib.fp8_block_gemm_gated_workspace
    assert f(8, 256, 384, 0, 1) > 0 and f(8, 200, 384, 0, 0) == -1 and f(-1, 256, 384, 0, 1) == -1 and f(8, 256, 384, 2, 0) == -1
    assert f(5000, 2048, 384, 0, 0) == f(5000, 2048, 384, 1, 0) == f(5000, 2048, 384, 0, 1) == 0
    assert g() in PASSED and g(gu=None) in PASSED and g(ht=1) in PASSED and g(act=1) in PASSED
    codes = dict(h=None, q=P[6], s=P[7])
    assert g(**codes) in PASSED and g(**codes, gu=None) in PASSED
    assert gated(lib, M=0, A=None) == OK
    assert g(act=2) == UNSUP and g(ht=2) == UNSUP and g(q=P[6], s=P[7]) == UNSUP
    for c in (dict(M=-1), dict(I=0), dict(I=200), dict(K=200), dict(K=0)):
        assert g(**c) == SHAPE, c
    assert g(I=1 << 18, K=1 << 13) == UNSUP and g(I=(1 << 24) + 128) == UNSUP and g(M=1 << 40) == UNSUP
    for k in ("A", "sA", "W", "s13"):
        assert g(**{k: None}) == NULL, k
    assert g(h=None) == NULL and g(h=None, q=P[6]) == NULL and g(h=None, s=P[7]) == NULL
    for k, v in (("lda", 368), ("ld_sa", M - 1), ("ld_s13", 2), ("ldh", 240), ("ld_gu", 496)):
        assert g(**{k: v}) == LD, k
    assert g(**codes, ldq=240) == LD and g(**codes, ld_s=M - 1) == LD
    for k in ("lda", "ldh", "ld_gu", "ld_sa", "ld_s13"):
        assert g(**{k: 1 << 50}) == UNSUP, k
    for k, v in (("lda", 392), ("ldh", 260), ("ld_gu", 516), ("A", P[0] + 8), ("W", P[2] + 8), ("sA", P[1] + 2), ("h", P[4] + 8),
                 ("gu", P[5] + 8), ("s13", P[3] + 1)):
        assert g(**{k: v}) == ALIGN, k
    assert g(**{**codes, "q": P[6] + 8}) == ALIGN and g(**codes, ldq=264) == ALIGN and g(**{**codes, "s": P[7] + 2}) == ALIGN
    for k, v in (("h", P[0]), ("h", P[1]), ("h", P[2] + 4096), ("gu", P[3]), ("gu", P[4] + 256)):
        assert g(**{k: v}) == ALIAS, (k, v)
    assert g(**{**codes, "q": P[5]}) == ALIAS and g(**{**codes, "s": P[6]}) == ALIAS and g(**{**codes, "s": P[1]}) == ALIAS
    for result, out in ((dict(), P[4]), (dict(ht=1), P[4]), (codes, P[6])):
        need = f(M, 256, 384, result.get("ht", 0), result is codes)
        if need > 0:
            few = {**result, "bytes": need}
            assert g(**few) in PASSED and g(**{**few, "bytes": need - 1}) == SHAPE
            assert g(**{**few, "ws": None}) == NULL and g(**{**few, "ws": P[9] + 4}) == ALIGN
            assert g(**{**few, "ws": P[0]}) == ALIAS and g(**{**few, "ws": out}) == ALIAS
        else:
            assert g(**result, ws=None, bytes=0) in PASSED


BACK = "T I dh ld_dh gu ld_gu act d ld_d q ldq s ld_s qt ldqt st ld_st ht sht ld_sht stream".split()


def back(lib, **c):
    base = dict(T=130, I=256, dh=P[0], ld_dh=256, gu=P[1], ld_gu=512, act=0, d=P[2], ld_d=512, q=P[3], ldq=512, s=P[4], ld_s=132,
                qt=P[5], ldqt=256, st=P[6], ld_st=512, ht=P[7], sht=P[8], ld_sht=256, stream=None)
    return call(lib.fp8_gated_backward, BACK, base, c)


def test_gated_backward_validation(lib):
    none = dict(d=None, q=None, s=None, qt=None, st=None, ht=None, sht=None)
    assert back(lib) in PASSED
    assert back(lib, **none) == NULL
    for keep in (("d",), ("q", "s"), ("qt", "st"), ("ht", "sht")):
        assert back(lib, **{k: v for k, v in none.items() if k not in keep}) in PASSED, keep
        if len(keep) == 2:
            for k in keep:
                assert back(lib, **{k: None}) == NULL, k
    assert back(lib, T=0, dh=None) == OK and back(lib, I=0, dh=None) == OK
    assert back(lib, act=-1) == UNSUP and back(lib, T=1 << 40) == UNSUP and back(lib, T=1 << 30, I=1 << 20) == UNSUP
    assert back(lib, T=-1) == SHAPE and back(lib, I=200) == SHAPE
    assert back(lib, dh=None) == NULL and back(lib, gu=None) == NULL
    for k, v in (("ld_dh", 248), ("ld_gu", 504), ("ld_d", 504), ("ldq", 496), ("ld_s", 129), ("ldqt", 128), ("ld_st", 511),
                 ("ld_sht", 255)):
        assert back(lib, **{k: v}) == LD, k
        assert back(lib, **{k: 1 << 60}) == UNSUP, k
    for k in ("ld_dh", "ld_gu", "ld_d", "ldq", "ldqt"):      # no overflow on the way
        assert back(lib, **{**dict(T=1 << 28, I=128, ldqt=1 << 28, ld_s=1 << 28), k: 1 << 40}) == UNSUP, k
    for k, v in (("ld_dh", 260), ("ld_gu", 516), ("ld_d", 516), ("ldq", 520), ("ldqt", 264)):
        assert back(lib, **{k: v}) == ALIGN, k
    for k in ("dh", "gu", "d", "q", "qt", "ht"):
        assert back(lib, **{k: P[12] + 8}) == ALIGN, k
    for k in ("s", "st", "sht"):
        assert back(lib, **{k: P[12] + 2}) == ALIGN, k
    for k, v in (("d", P[0]), ("q", P[1] + 1024), ("qt", P[0]), ("ht", P[1]), ("s", P[3]), ("st", P[4]), ("sht", P[7]), ("ht", P[5])):
        assert back(lib, **{k: v}) == ALIAS, (k, v)


COLS = "x rows cols ldx q s ld_s stream".split()


def cols(lib, **c):
    base = dict(x=P[0], rows=130, cols=256, ldx=256, q=P[1], s=P[2], ld_s=256, stream=None)
    return call(lib.fp8_quant_act_cols, COLS, base, c)


def test_quant_act_cols_validation(lib):
    assert cols(lib) in PASSED and cols(lib, rows=0, x=None) == OK and cols(lib, cols=0, x=None) == OK
    assert cols(lib, rows=-1) == SHAPE and cols(lib, cols=200) == SHAPE and cols(lib, rows=1 << 40) == UNSUP
    for k in ("x", "q", "s"):
        assert cols(lib, **{k: None}) == NULL
    for k in ("ldx", "ld_s"):
        assert cols(lib, **{k: 248}) == LD and cols(lib, **{k: 1 << 60}) == UNSUP
    for k, v in (("x", P[0] + 2), ("q", P[1] + 8), ("s", P[2] + 2), ("ldx", 260)):
        assert cols(lib, **{k: v}) == ALIGN
    assert cols(lib, rows=1 << 28, cols=128, ldx=1 << 40) == UNSUP      # no overflow on the way
    assert cols(lib, q=P[0]) == ALIAS and cols(lib, s=P[0]) == ALIAS and cols(lib, s=P[1] + 256) == ALIAS
    assert cols(lib, s=P[1] + 256 * 256 - 4) == ALIAS    # the padded columns of codes count


HEADS = "T dim xt q k wt norm eps rot pos pbytes axes sections freq adjacent stream".split()


def heads(lib, q=None, k=None, **c):
    from fine_grained_fp8_amd import _lib
    hq = {**dict(x=P[0], heads=4, ld_token=8 * 64, ld_head=64, weight=P[1], y=P[2], ldy_token=4 * 64, ldy_head=64), **(q or {})}
    hk = {**dict(x=P[0] + 4 * 64 * 2, heads=2, ld_token=8 * 64, ld_head=64, weight=P[1], y=P[3], ldy_token=2 * 64, ldy_head=64),
          **(k or {})}
    sec = c.pop("sections", None)
    base = dict(T=10, dim=64, xt=0, q=ctypes.byref(_lib.Heads(**hq)), k=ctypes.byref(_lib.Heads(**hk)), wt=0, norm=1, eps=1e-6,
                rot=64, pos=P[4], pbytes=8, axes=1, sections=None if sec is None else (ctypes.c_int64 * len(sec))(*sec),
                freq=P[5], adjacent=0, stream=None)
    for name, h in (("q", q), ("k", k)):
        if h is False:
            base[name] = None
    return call(lib.fp8_head_norm_rotary, HEADS, base, c)


def test_head_norm_rotary_validation(lib):
    assert heads(lib) in PASSED and heads(lib, k=False) in PASSED and heads(lib, q=False) in PASSED
    assert heads(lib, q=False, k=False) == SHAPE and heads(lib, q=dict(heads=0), k=dict(heads=0)) == SHAPE
    assert heads(lib, k=dict(heads=0, x=None, y=None)) in PASSED
    assert heads(lib, rot=0, pos=None, freq=None) in PASSED and heads(lib, rot=20) in PASSED
    assert heads(lib, axes=3, sections=[16, 8, 8]) in PASSED and heads(lib, axes=3, sections=[32, 0, 0]) in PASSED
    assert heads(lib, T=0, pos=None, freq=None, q=dict(x=None, y=None)) == OK
    for c in (dict(T=-1), dict(dim=0), dict(dim=63), dict(rot=66), dict(rot=7), dict(rot=-2), dict(eps=-1.0),
              dict(eps=float("nan")), dict(axes=2, sections=[16, 8]), dict(axes=2, sections=[33, -1]), dict(axes=1, sections=[31])):
        assert heads(lib, **c) == SHAPE, c
    assert heads(lib, q=dict(heads=-1)) == SHAPE
    for c in (dict(xt=2), dict(wt=2), dict(norm=3), dict(dim=1026), dict(T=1 << 40), dict(axes=0), dict(axes=5, sections=[32, 0, 0, 0, 0]),
              dict(pbytes=2), dict(norm=0)):      # norm 0 with weights
        assert heads(lib, **c) == UNSUP, c
    for n in ("ld_token", "ldy_token"):                       # no overflow on the way
        assert heads(lib, T=1 << 25, q={n: 1 << 40}) == UNSUP, n
    assert heads(lib, q=dict(heads=1 << 20, ld_head=1 << 40)) == UNSUP
    assert heads(lib, T=1, q=dict(ld_token=1 << 44)) in PASSED
    assert heads(lib, norm=0, q=dict(weight=None), k=dict(weight=None)) in PASSED
    assert heads(lib, q=dict(heads=1 << 30)) == UNSUP and heads(lib, q=dict(ld_token=1 << 60)) == UNSUP
    for c in (dict(pos=None), dict(freq=None), dict(axes=2), dict(q=dict(x=None)), dict(k=dict(y=None))):
        assert heads(lib, **c) == NULL, c
    for c in (dict(ld_head=63), dict(ld_token=255), dict(ldy_head=32), dict(ldy_token=4 * 64 - 1), dict(ldy_token=-256), dict(ld_head=0)):
        assert heads(lib, q=c) == LD, c
    # head by head, and one token or one head whose other stride does not matter
    assert heads(lib, q=dict(ld_token=64, ld_head=640, x=P[6], ldy_token=64, ldy_head=640)) in PASSED
    assert heads(lib, q=dict(ld_token=64, ld_head=639, x=P[6])) == LD
    assert heads(lib, T=1, q=dict(ld_token=0), k=dict(ld_token=5)) in PASSED
    assert heads(lib, q=dict(heads=1, ld_head=0, ldy_head=7, x=P[6])) in PASSED
    for c in (dict(pos=P[4] + 4), dict(freq=P[5] + 4), dict(q=dict(x=P[0] + 1)), dict(q=dict(y=P[2] + 1)), dict(q=dict(weight=P[1] + 1)),
              dict(wt=1, q=dict(weight=P[1] + 2)), dict(xt=1, q=dict(x=P[6] + 2))):
        assert heads(lib, **c) == ALIGN, c
    assert heads(lib, pos=P[4] + 4, pbytes=4) in PASSED
    for c in (dict(q=dict(y=P[0])), dict(k=dict(y=P[0] + 64)), dict(q=dict(y=P[1])), dict(k=dict(y=P[4])), dict(q=dict(y=P[5] + 2)),
              dict(k=dict(y=P[2] + 128))):
        assert heads(lib, **c) == ALIAS, c
    # both outputs side by side in each token's row; sharing a channel; the next row's first
    side = dict(ldy_token=6 * 64)
    assert heads(lib, q=side, k=dict(side, y=P[2] + 4 * 64 * 2)) in PASSED
    assert heads(lib, q=dict(side, y=P[2] + 2 * 64 * 2), k=dict(side, y=P[2])) in PASSED
    assert heads(lib, q=side, k=dict(side, y=P[2] + 4 * 64 * 2 - 2)) == ALIAS
    assert heads(lib, q=side, k=dict(side, y=P[2] + 4 * 64 * 2 + 2)) == ALIAS
    assert heads(lib, q=side, k=dict(ldy_token=7 * 64, y=P[2] + 4 * 64 * 2)) == ALIAS


HBACK = "T dim xt q k wt norm eps rot pos pbytes axes sections freq adjacent ws bytes stream".split()


def hback(lib, q=None, k=None, **c):
    from fine_grained_fp8_amd import _lib
    hq = {**dict(x=P[0], heads=4, ld_token=256, ld_head=64, weight=P[1], dy=P[2], lddy_token=256, lddy_head=64, dx=P[3],
                 lddx_token=256, lddx_head=64, dweight=P[4]), **(q or {})}
    hk = {**dict(x=P[5], heads=2, ld_token=128, ld_head=64, weight=P[1], dy=P[6], lddy_token=128, lddy_head=64, dx=P[7],
                 lddx_token=128, lddx_head=64, dweight=P[8]), **(k or {})}
    base = dict(T=10, dim=64, xt=1, q=ctypes.byref(_lib.HeadsGrad(**hq)), k=ctypes.byref(_lib.HeadsGrad(**hk)), wt=1, norm=2,
                eps=1e-6, rot=64, pos=P[9], pbytes=4, axes=1, sections=None, freq=P[10], adjacent=1, ws=P[11], bytes=1 << 24,
                stream=None)
    for name, h in (("q", q), ("k", k)):
        if h is False:
            base[name] = None
    return call(lib.fp8_head_norm_rotary_backward, HBACK, base, c)


def test_head_norm_rotary_backward_validation(lib):
    f = lib.fp8_head_norm_rotary_backward_workspace
    assert f(10, 4, 2, 64) > 0 and f(0, 4, 2, 64) == 0 and f(10, 0, 0, 64) == -1 and f(10, 4, 2, 63) == -1 and f(-1, 4, 2, 64) == -1
    assert hback(lib) in PASSED and hback(lib, q=False) in PASSED and hback(lib, k=False) in PASSED
    assert hback(lib, q=dict(dweight=None, weight=None)) in PASSED
    no = dict(weight=None, dweight=None, x=None, ld_token=-5)
    assert hback(lib, norm=0, q=no, k=no, ws=None, bytes=0) in PASSED
    assert hback(lib, norm=0, q=no) == UNSUP and hback(lib, norm=0, q=no, k=dict(no, dweight=P[8])) == UNSUP
    assert hback(lib, T=0, q=dict(dweight=None), k=dict(dweight=None), ws=None) == OK
    empty = dict(heads=0, x=None, dy=None, dx=None, weight=None)     # its dweight is written all the same
    assert hback(lib, k=empty) in PASSED and hback(lib, k=dict(empty, dweight=None)) in PASSED
    assert hback(lib, norm=0, q=no, k=empty) == UNSUP and hback(lib, k=dict(empty, dweight=P[8] + 2)) == ALIGN
    assert hback(lib, k=dict(empty, dweight=P[0])) == ALIAS and hback(lib, k=dict(empty, dweight=P[4])) == ALIAS
    for c in (dict(ws=None), dict(q=dict(x=None)), dict(q=dict(dy=None)), dict(k=dict(dx=None)), dict(pos=None)):
        assert hback(lib, **c) == NULL, c
    assert hback(lib, bytes=100) == SHAPE and hback(lib, dim=62, rot=64) == SHAPE
    for n in ("ld_token", "lddy_token", "lddx_token", "ld_head", "lddy_head", "lddx_head"):
        assert hback(lib, q={n: 60}) == LD, n
        assert hback(lib, q={n: 1 << 60}) == UNSUP, n
    for n in ("x", "dy", "dx", "weight", "dweight"):
        assert hback(lib, q={n: P[12] + 2}) == ALIGN, n
    for n in ("ld_token", "lddy_token", "lddx_token"):
        assert hback(lib, T=1 << 25, q={n: 1 << 40}) == UNSUP, n
    assert hback(lib, ws=P[11] + 8) == ALIGN
    for c in (dict(q=dict(dx=P[0])), dict(q=dict(dx=P[6])), dict(q=dict(dx=P[7])), dict(k=dict(dx=P[10])), dict(q=dict(dweight=P[9])),
              dict(k=dict(dweight=P[4] + 4)), dict(q=dict(dweight=P[1])), dict(ws=P[0]), dict(ws=P[1]), dict(ws=P[3]), dict(ws=P[8]),
              dict(ws=P[6] + 16), dict(k=dict(dweight=P[3] + 512)), dict(ws=P[9])):
        assert hback(lib, **c) == ALIAS, c


def test_sizes_of_every_workspace_have_an_answer(tmp_path):
    """The size rules of the built library over their range, an empty batch among them, in a
    process of their own (an integer division by zero there ends it)."""
    from fine_grained_fp8_amd import _lib, build
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    code = """
from fine_grained_fp8_amd import _lib
lib = _lib.load_library()
f, g = lib.fp8_block_gemm_gated_workspace, lib.fp8_head_norm_rotary_backward_workspace
for I in (128, 2048, 8064, 8192, 8320, 18432, 24576, (1 << 24) - 256):
    for K in (128, 1024, 7168, 16384, (1 << 23) - 128):
        fits = (I + 128) * K < 1 << 31
        for h_dtype, codes in ((0, 0), (1, 0), (0, 1)):
            print("I", I, "K", K, h_dtype, codes, flush=True)
            assert f(0, I, K, h_dtype, codes) == (0 if fits else -1)
            for M in (1, 16, 17, 64, 65, 128, 1333, 4096, 42000, 1 << 31):
                n = f(M, I, K, h_dtype, codes)
                unit = M * I * 4
                assert n == -1 if not fits or M * I // 16384 >= 1 << 31 else n >= 0 and n % unit == 0, (M, n)
for T in (0, 1, 3, 4096, 1 << 25):
    for q in (0, 1, 64, 1 << 20):
        for k in (0, 1, 64, 1 << 20):
            for dim in (2, 64, 130, 1024):
                n = g(T, q, k, dim)
                print("T", T, q, k, dim, n, flush=True)
                assert n == -1 if q + k == 0 else n == 0 if T == 0 else 0 < n <= 1280 * dim * 4
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stdout[-200:], r.stderr[-2000:])


def test_size_rules_under_ubsan(tmp_path):
    """block_rules.hpp built on the host with the undefined-behaviour sanitizer (divisions
    by zero and overflows end it), swept over the sizes that the checks let through."""
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("g++ is not available")
    exe = str(tmp_path / "check_block_rules")
    r = subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=undefined", "-fno-sanitize-recover=undefined",
                        "-I", os.path.join(ROOT, "fine_grained_fp8_amd", "csrc"), os.path.join(ROOT, "tests", "c", "check_block_rules.cpp"),
                        "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.endswith("violations=0\n"), r.stdout[-500:] + r.stderr[-2000:]


def test_block_validation_under_asan_ubsan(tmp_path):
    """api_blocks.cpp built on the host with sanitizers, its launchers
    replaced by stubs, runs the validation tests above without a report."""
    if os.environ.get("FP8BS_SANITIZED_BLOCKS"):
        pytest.skip("already the sanitized child run")
    gxx = shutil.which("g++")
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    if not gxx or not os.path.exists(os.path.join(rocm, "include", "hip", "hip_runtime.h")):
        pytest.skip("g++ or the HIP headers are not available")
    so = str(tmp_path / "libblocks_san.so")
    csrc = os.path.join(ROOT, "fine_grained_fp8_amd", "csrc")
    r = subprocess.run([gxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined",
                        "-fno-omit-frame-pointer", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__",
                        "-I", os.path.join(rocm, "include"), "-I", os.path.join(ROOT, "include"), "-I", csrc,
                        os.path.join(csrc, "api_blocks.cpp"), os.path.join(ROOT, "tests", "c", "block_stubs.cpp"),
                        "-L", os.path.join(rocm, "lib"), "-Wl,-rpath," + os.path.join(rocm, "lib"), "-lamdhip64", "-o", so],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    asan = subprocess.run([gxx, "-print-file-name=libasan.so"], capture_output=True, text=True).stdout.strip()
    env = dict(os.environ, LD_PRELOAD=asan, FP8BS_SANITIZED_BLOCKS=so, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([sys.executable, "-m", "pytest", os.path.abspath(__file__), "-q", "-x", "-p", "no:cacheprovider",
                        "-k", "validation and not asan"], env=env, capture_output=True, text=True, timeout=600, cwd=ROOT)
    report = r.stdout[-3000:] + r.stderr[-3000:]
    assert r.returncode == 0 and " passed" in r.stdout, report
    assert "AddressSanitizer" not in r.stderr and "runtime error" not in r.stderr, report
