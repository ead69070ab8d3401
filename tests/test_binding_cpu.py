"""The binding's own work (ops.py), on the CPU: a stand-in library records the
calls, and streams and the memory pool are recorded instead of used."""
import contextlib
import types

import pytest
import torch

from fine_grained_fp8_amd import ops


class Recorder:
    """Which stream was current at each allocation, and which streams each
    tensor was reported to."""

    def __init__(self, monkeypatch):
        self.current = types.SimpleNamespace(cuda_stream=1)
        self.side = types.SimpleNamespace(cuda_stream=2)
        self.born, self.told, self.calls = {}, {}, []
        self.keep = []          # no address comes back within a test
        for name in ("empty", "full"):
            monkeypatch.setattr(torch, name, self.tracked(getattr(torch, name)))
        monkeypatch.setattr(torch, "empty_like", self.tracked(torch.empty_like))
        monkeypatch.setattr(torch.Tensor, "record_stream",
                            lambda t, s: self.told.setdefault(t.data_ptr(), []).append(s.cuda_stream), raising=False)
        monkeypatch.setattr(torch.cuda, "stream", self.use)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self.current)
        monkeypatch.setattr(ops, "_stream", lambda s=None: (self.current if s is None else s).cuda_stream)
        for check in ("_check_2d", "_check_vec"):
            monkeypatch.setattr(ops, check, lambda *a, **k: None)
        monkeypatch.setattr(ops._lib, "load_library", lambda path=None: self)

    def tracked(self, make):
        def made(*args, **kwargs):
            t = make(*args, **kwargs)
            self.born[t.data_ptr()] = self.current.cuda_stream
            self.keep.append(t)
            return t
        return made

    @contextlib.contextmanager
    def use(self, stream):
        before, self.current = self.current, stream or self.current
        yield
        self.current = before

    def __getattr__(self, name):
        if not name.startswith("fp8_"):
            raise AttributeError(name)

        def entry(*args):
            if name.endswith("_workspace"):
                return 4096
            self.calls.append((name, args))
            return 0
        return entry


@pytest.fixture
def rec(monkeypatch):
    return Recorder(monkeypatch)


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def codes(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def scales(*shape):
    return torch.ones(shape)


LAYER_CALLS = {
    "layer_norm": lambda **k: ops.layer_norm(bf16(4, 256), return_stats=True, **k),
    "layer_norm_quant": lambda **k: ops.layer_norm_quant(bf16(4, 256), return_y=True, return_stats=True, **k),
    "layer_norm_backward": lambda **k: ops.layer_norm_backward(bf16(4, 256), bf16(4, 256), scales(4), scales(4), **k),
    "moe_few_tokens": lambda **k: ops.moe_few_tokens(bf16(4, 256), bf16(8, 256), codes(2, 256, 256), scales(2, 2, 2),
                                                     codes(2, 256, 128), scales(2, 2, 1), top_k=2, return_routing=True, **k),
    "adapter_linear": lambda **k: ops.adapter_linear(bf16(4, 256), codes(384, 256), scales(3, 2), bf16(3, 16, 256),
                                                     bf16(3, 384, 16), torch.zeros(4, dtype=torch.int32), **k),
}
SCRATCH = {"layer_norm_backward", "moe_few_tokens", "adapter_linear"}


def check_memory_of_a_call(rec, call, scratch):
    """On a stream that is not the current one a call's memory comes from that
    stream's pool: memory of the current stream's pool may still be in use by
    work that the current stream has pending (a former call's scratch is free
    to the pool as soon as that call returned)."""
    before = set(rec.born)
    out = call(stream=rec.side)
    out = [t for t in (out if isinstance(out, tuple) else (out,)) if t is not None]
    new = set(rec.born) - before
    (_, args), = rec.calls
    assert args[-1] == 2
    used = {a for a in args if a in new}
    assert {t.data_ptr() for t in out} <= used
    assert all(rec.born[a] == 2 for a in used), {a: rec.born[a] for a in used}
    # the caller's later work on the current stream holds an output's memory back
    assert all(1 in rec.told.get(t.data_ptr(), []) for t in out)
    assert len(used) == len(out) + scratch
    assert rec.current.cuda_stream == 1


@pytest.mark.parametrize("name", LAYER_CALLS)
def test_memory_of_a_call_on_another_stream(rec, name):
    check_memory_of_a_call(rec, LAYER_CALLS[name], int(name in SCRATCH))


@pytest.mark.parametrize("name", LAYER_CALLS)
def test_memory_of_a_call_on_the_current_stream(rec, name):
    for kwargs in ({}, {"stream": rec.current}):
        LAYER_CALLS[name](**kwargs)
    assert all(args[-1] == 1 for _, args in rec.calls)
    assert set(rec.born.values()) == {1} and not rec.told


BASE_CALLS = {
    "quant_act_1x128": lambda **k: ops.quant_act_1x128(bf16(4, 256), return_amax=True, **k),
    "quant_act_dual": lambda **k: ops.quant_act_dual(bf16(128, 256), **k),
    "quant_act_dual_tiled": lambda **k: ops.quant_act_dual(bf16(128, 256), tiled=True, **k),
    "quant_weight_128x128": lambda **k: ops.quant_weight_128x128(bf16(128, 256), transposed=True, **k),
    "quant_weight_128x128_tiled": lambda **k: ops.quant_weight_128x128(bf16(128, 256), tiled=True, transposed=True, **k),
    "block_gemm": lambda **k: ops.block_gemm("fprop", codes(4, 256), scales(2, 4), codes(128, 256), scales(1, 2), **k),
    "block_gemm_fused_quant": lambda **k: ops.block_gemm_fused_quant(bf16(4, 256), codes(128, 256), scales(1, 2),
                                                                     with_codes=True, **k),
    "block_gemm_grouped": lambda **k: ops.block_gemm_grouped(torch.zeros(3, dtype=torch.int32), codes(4, 256), scales(2, 4),
                                                             codes(2, 128, 256), scales(2, 1, 2), **k),
    "cast_e4m3": lambda **k: ops.cast_e4m3(scales(64), **k),
    "pack_tokens": lambda **k: ops.pack_tokens(bf16(4, 256), **k),
    "unpack_tokens": lambda **k: ops.unpack_tokens(codes(4, 272), 256, **k),
    "dequant_tokens": lambda **k: ops.dequant_tokens(codes(4, 272), 256, **k),
    "gemm_promotion": lambda **k: ops.gemm_promotion(codes(4, 256), codes(128, 256), 128, **k),
    "probe_mfma": lambda **k: ops.probe_mfma(codes(4096), 2, 1, **k),
    "probe_recip_online": lambda **k: ops.probe_recip_online(scales(64), **k),
    "quant_act_tiles": lambda **k: ops.quant_act_tiles(bf16(4, 256), **k),
}


@pytest.mark.parametrize("name", BASE_CALLS)
def test_outputs_of_the_other_calls_on_another_stream(rec, name, monkeypatch):
    monkeypatch.setattr(torch.Tensor, "is_cuda", True, raising=False)
    check_memory_of_a_call(rec, BASE_CALLS[name], 0)


@pytest.mark.parametrize("side", [False, True])
def test_statistics_of_rows_without_columns(rec, side, monkeypatch):
    """Without columns the library writes nothing: sum / 0 is NaN, and so are
    both statistics (on the call's stream)."""
    filled = []
    fill = torch.Tensor.fill_
    monkeypatch.setattr(torch.Tensor, "fill_", lambda t, v: (filled.append(rec.current.cuda_stream), fill(t, v))[1])
    real = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: fill(real(*a, **k), 7))
    stream = rec.side if side else None
    for out in (ops.layer_norm(bf16(4, 0), return_stats=True, stream=stream),
                ops.layer_norm_quant(bf16(4, 0), return_stats=True, stream=stream)):
        mean, rstd = out[-2:]
        assert mean.shape == rstd.shape == (4,) and mean.isnan().all() and rstd.isnan().all()
    assert filled == [2 if side else 1] * 4


@pytest.mark.parametrize("name", ["moe_few_tokens", "adapter_linear"])
def test_output_types_that_the_library_does_not_write(rec, name):
    """Refused: the library writes bfloat16 or float32, and another type's
    tensor would hold its bits."""
    for dtype in (torch.float16, torch.float64, torch.int16):
        with pytest.raises(TypeError):
            LAYER_CALLS[name](out_dtype=dtype)
    assert not rec.calls
    for dtype in (torch.bfloat16, torch.float32):
        assert LAYER_CALLS[name](out_dtype=dtype) is not None


def test_a_library_named_by_path_has_whole_parts_of_the_abi(tmp_path, monkeypatch):
    """A build that lacks single entry points (a stale one) is refused when it is
    loaded, not at the first call; one that holds the entry points of one source
    file, as the host-only builds of the validation code do, is taken."""
    import shutil
    import subprocess
    from fine_grained_fp8_amd import _lib
    gcc = shutil.which("gcc")
    if not gcc:
        pytest.skip("no C compiler")

    def load(names):
        src, so = tmp_path / "stub.c", tmp_path / f"lib{len(list(tmp_path.iterdir()))}.so"     # a name of its own
        src.write_text("\n".join(f"int {n}(void) {{ return 0; }}" for n in names))
        subprocess.run([gcc, "-shared", "-fPIC", "-o", str(so), str(src)], check=True)
        monkeypatch.setattr(_lib, "_lib", None)
        return _lib.load_library(str(so))

    layers = [n for n in _lib.SIGNATURES if n in _lib.LAYER_ENTRIES]
    base = [n for n in _lib.SIGNATURES if n not in _lib.LAYER_ENTRIES]
    assert set(_lib.LAYER_ENTRIES) <= set(_lib.SIGNATURES) and len(layers) == 7
    for names in (base + layers, base, layers):
        lib = load(names)
        assert all(hasattr(lib, n) for n in names)
    for names in (base[1:] + layers, base + layers[:-1], base[:-1], layers[1:], []):
        with pytest.raises(RuntimeError, match="lacks"):
            load(names)
        assert _lib._lib is None
