"""The binding's work for the operators between the FP8 products, on the CPU: the
memory of a call on another stream, refusals of types and devices, parts of the
ABI in a library named by path."""
import ctypes
import shutil
import subprocess

import pytest
import torch

from fine_grained_fp8_amd import _lib, ops
from test_binding_cpu import Recorder, bf16, codes, scales


@pytest.fixture
def rec(monkeypatch):
    monkeypatch.setattr(torch.Tensor, "is_cuda", True, raising=False)     # the stand-ins pass as device tensors
    monkeypatch.setattr(ops, "_on_current_device", lambda *a: None)
    ops._gated_workspace.cache_clear()
    ops._heads_workspace.cache_clear()
    yield Recorder(monkeypatch)
    ops._gated_workspace.cache_clear()
    ops._heads_workspace.cache_clear()


ROTARY = dict(positions=torch.arange(4), freq=torch.ones(32, dtype=torch.float64))
CALLS = {   # call, scratch allocations
    "block_gemm_gated": (lambda **k: ops.block_gemm_gated(codes(4, 256), scales(2, 4), codes(512, 256), scales(4, 2),
                                                          return_gate_up=True, **k), 1),
    "block_gemm_gated_quant": (lambda **k: ops.block_gemm_gated_quant(codes(4, 256), scales(2, 4), codes(512, 256), scales(4, 2),
                                                                      return_gate_up=True, **k), 1),
    "gated_backward": (lambda **k: ops.gated_backward(bf16(4, 128), bf16(4, 256), **k), 0),
    "gated_backward_quant": (lambda **k: ops.gated_backward_quant(bf16(4, 128), bf16(4, 256), return_h=True, **k), 0),
    "quant_act_cols": (lambda **k: ops.quant_act_cols(bf16(4, 128), **k), 0),
    "head_norm_rotary": (lambda **k: ops.head_norm_rotary(bf16(4, 2, 64), bf16(4, 1, 64), **ROTARY, **k), 0),
    "head_norm_rotary_backward": (lambda **k: ops.head_norm_rotary_backward(bf16(4, 2, 64), bf16(4, 1, 64), bf16(4, 2, 64),
                                                                            bf16(4, 1, 64), **ROTARY, **k), 1),
}


def addresses(args):
    """Those given directly, and those inside of fp8_heads structures."""
    for a in args:
        if isinstance(a, int):
            yield a
        elif isinstance(a, ctypes.Structure):
            yield from (getattr(a, n) for n, t in a._fields_ if t is ctypes.c_void_p)


@pytest.mark.parametrize("name", CALLS)
def test_memory_of_a_call_on_another_stream(rec, name):
    call, scratch = CALLS[name]
    before = set(rec.born)
    out = call(stream=rec.side)
    out = list(out) if isinstance(out, tuple) else [out]
    new = set(rec.born) - before
    (_, args), = rec.calls
    assert args[-1] == 2
    used = {a for a in addresses(args) if a in new}
    assert {t.data_ptr() for t in out} <= used
    assert all(rec.born[a] == 2 for a in used)
    assert all(1 in rec.told.get(t.data_ptr(), []) for t in out)
    assert len(used) == len(out) + scratch


@pytest.mark.parametrize("name", CALLS)
def test_memory_of_a_call_on_the_current_stream(rec, name):
    for kwargs in ({}, {"stream": rec.current}):
        CALLS[name][0](**kwargs)
    assert all(args[-1] == 1 for _, args in rec.calls)
    assert set(rec.born.values()) == {1} and not rec.told


def test_tensors_of_another_device_than_the_current_one(monkeypatch):
    """Refused before anything is launched."""
    class Elsewhere:
        device = torch.device("cuda", 1)

        def get_device(self):
            return 1
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="current device"):
        ops._on_current_device("x", Elsewhere())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    ops._on_current_device("x", Elsewhere())


def test_gated_output_types(rec):
    for dtype in (torch.float16, torch.float64, torch.int16):
        with pytest.raises(TypeError):
            CALLS["block_gemm_gated"][0](out_dtype=dtype)
    assert not rec.calls


def test_a_library_named_by_path_may_hold_these_entry_points_alone(tmp_path, monkeypatch):
    gcc = shutil.which("gcc")
    if not gcc:
        pytest.skip("no C compiler")

    def load(names):
        src, so = tmp_path / "stub.c", tmp_path / f"lib{len(list(tmp_path.iterdir()))}.so"
        src.write_text("\n".join(f"int {n}(void) {{ return 0; }}" for n in names))
        subprocess.run([gcc, "-shared", "-fPIC", "-o", str(so), str(src)], check=True)
        monkeypatch.setattr(_lib, "_lib", None)
        return _lib.load_library(str(so))

    mine = sorted(_lib.BLOCK_ENTRIES)
    layers = sorted(_lib.LAYER_ENTRIES)
    core = sorted(set(_lib.SIGNATURES) - _lib.BLOCK_ENTRIES - _lib.LAYER_ENTRIES)
    assert len(mine) == 7 and not _lib.BLOCK_ENTRIES & _lib.LAYER_ENTRIES
    for names in (mine, core, mine + layers, core + layers):
        assert all(hasattr(load(names), n) for n in names)
    for names in (mine[1:], core + mine[1:], core[1:] + mine):
        with pytest.raises(RuntimeError, match="lacks"):
            load(names)
