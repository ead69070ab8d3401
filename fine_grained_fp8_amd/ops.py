"""Thin PyTorch-facing binding of libfp8bs.so (argument marshalling only).

Tensors are used for device memory and the current HIP stream; every step of
the computation runs in the library's kernels.  Names follow the C ABI in
include/fp8bs.h.  Scale arrays are MN-major: [K/128][ld] with
ld = round_up(rows, 4) for 1x128 row tiles.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _lib

FP8_DTYPE = torch.uint8


def _stream(stream=None) -> int:
    if stream is not None:
        return stream.cuda_stream
    # the raw handle: building the Stream object takes longer than a short
    # kernel's launch (2.8 us against 0.1 us)
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _empty(shape, dtype, device, stream, scratch=False):
    """Uninitialized memory for a call on `stream` (None: the current one).

    It comes from the pool of the stream that the kernels run on: a block of
    the current stream's pool may still be in use by work pending there (a
    former call's scratch goes back to the pool when that call returns), which
    a kernel on another stream would not wait for.  What the call returns is
    the caller's to read on the current stream, so that stream's work holds
    the memory back when the tensor is dropped; scratch is seen by `stream`
    alone."""
    if stream is None or stream.cuda_stream == _stream():
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if not scratch:
        t.record_stream(current)
    return t


def _empty_as(x, stream):
    """A contiguous tensor of x's shape and type (the short call where x is one)."""
    if stream is None and x.is_contiguous():
        return torch.empty_like(x)
    return _empty(x.shape, x.dtype, x.device, stream)


def _workspace(nbytes: int, device, stream):
    """Scratch memory of one call (nbytes -1: the call itself refuses)."""
    return _empty(max(nbytes, 0), torch.uint8, device, stream, scratch=True)


def _ptr(t):
    return None if t is None else ctypes_ptr(t)


def ctypes_ptr(t: torch.Tensor) -> int:
    return t.data_ptr()


def _check_2d(name, t, dtypes):
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name}: expected a 2-D row-major tensor, got shape {tuple(t.shape)} "
                         f"strides {t.stride()}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a device tensor")


def round_up(x: int, m: int) -> int:
    return (x + m - 1) // m * m


_BF16 = (torch.bfloat16, torch.int16, torch.uint16)


def quant_act_1x128(x: torch.Tensor, direction: str = "row", *, scales_in=None,
                    return_amax: bool = False, sat_count=None, out=None, scales_out=None, stream=None):
    """Online FP8 quantization of activations.

    direction "row": 1x128 tiles along each row; returns
        q [rows][cols] uint8, scales [cols/128][round_up(rows, 4)] float32.
    direction "col": 128x1 tiles along each column, transposed output; returns
        q [cols][rows] uint8, scales [rows/128][round_up(cols, 4)] float32.
    direction "col_tiled": as "col" with q holding the operand-tiled bytes of
        the transposed codes (for the "wgrad_tiled" GEMM layout).
    scales_in (row only): caller scales in the scale layout; then the returned
    scales are None.  return_amax adds the per-tile max |x| (same layout).
    sat_count: optional int32/uint32 device tensor of one element, incremented.
    out / scales_out: optional caller buffers for q (the shape above, uint8)
    and the scales (at least the shape above, float32, row-major; its row
    stride is passed as ld_s), so that repeated calls allocate nothing.
    Returns (q, scales, amax_or_None).
    """
    lib = _lib.load_library()
    _check_2d("x", x, _BF16)
    rows, cols = x.shape
    dev = x.device
    if direction == "row":
        q_shape = (rows, cols)
        s_shape = (cols // 128, round_up(rows, 4))
        tile_dir = _lib.TILE_ROW
    elif direction in ("col", "col_tiled"):
        q_shape = (cols, rows)
        s_shape = (rows // 128, round_up(cols, 4))
        tile_dir = _lib.TILE_COL if direction == "col" else _lib.TILE_COL_TILED
    else:
        raise ValueError(direction)
    if out is None:
        q = _empty(q_shape, torch.uint8, dev, stream)
    else:
        _check_2d("out", out, (torch.uint8, torch.float8_e4m3fn))
        if tuple(out.shape) != q_shape or not out.is_contiguous():
            raise ValueError(f"out: expected a contiguous {q_shape} tensor, got {tuple(out.shape)}")
        q = out
    if scales_in is not None:
        _check_2d("scales_in", scales_in, (torch.float32,))
        scales = None
        ld_s = scales_in.stride(0)
    elif scales_out is not None:
        _check_2d("scales_out", scales_out, (torch.float32,))
        if scales_out.shape[0] < s_shape[0] or scales_out.shape[1] < s_shape[1]:
            raise ValueError(f"scales_out: expected at least {s_shape}, got {tuple(scales_out.shape)}")
        scales = scales_out
        ld_s = scales_out.stride(0)
    else:
        scales = _empty(s_shape, torch.float32, dev, stream)
        ld_s = s_shape[1]
    amax = _empty(s_shape if scales_in is None else tuple(scales_in.shape), torch.float32, dev, stream) if return_amax else None
    st = lib.fp8_quant_act_1x128(
        _ptr(x), rows, cols, x.stride(0), tile_dir, _ptr(q), q.stride(0),
        _ptr(scales), ld_s, _ptr(scales_in), _ptr(amax), _ptr(sat_count), _stream(stream))
    _lib.check("fp8_quant_act_1x128", st)
    return q, scales, amax


def quant_act_dual(x: torch.Tensor, *, tiled: bool = False, stream=None):
    """Both orientations of x [rows][cols] BF16 from one read.

    Returns (q_row [rows][cols], s_row [cols/128][round_up(rows, 4)],
             q_col [cols][rows], s_col [rows/128][round_up(cols, 4)]) - the outputs of
    quant_act_1x128(x, "row") and quant_act_1x128(x, "col") ("col_tiled" if tiled).
    """
    lib = _lib.load_library()
    _check_2d("x", x, _BF16)
    rows, cols = x.shape
    q_row = _empty((rows, cols), torch.uint8, x.device, stream)
    s_row = _empty((cols // 128, round_up(rows, 4)), torch.float32, x.device, stream)
    q_col = _empty((cols, rows), torch.uint8, x.device, stream)
    s_col = _empty((rows // 128, round_up(cols, 4)), torch.float32, x.device, stream)
    if tiled:
        st = lib.fp8_quant_act_dual_tiled(_ptr(x), rows, cols, x.stride(0), _ptr(q_row), q_row.stride(0),
                                          _ptr(s_row), s_row.stride(0), _ptr(q_col), _ptr(s_col),
                                          s_col.stride(0), _stream(stream))
        _lib.check("fp8_quant_act_dual_tiled", st)
        return q_row, s_row, q_col, s_col
    st = lib.fp8_quant_act_dual(_ptr(x), rows, cols, x.stride(0), _ptr(q_row), q_row.stride(0),
                                _ptr(s_row), s_row.stride(0), _ptr(q_col), q_col.stride(0),
                                _ptr(s_col), s_col.stride(0), _stream(stream))
    _lib.check("fp8_quant_act_dual", st)
    return q_row, s_row, q_col, s_col


def quant_weight_128x128(w: torch.Tensor, *, transposed: bool = False, tiled: bool = False,
                         stream=None):
    """128x128 block quantization of weights [N][K].

    Returns (q [N][K] uint8, scales [N/128][K/128] float32, q_t [K][N] or None).
    tiled: q (and q_t) hold the operand-tiled bytes of the same codes, for
    the "fprop_tiled" / "dgrad_t_tiled" GEMM layouts (same shapes).
    """
    lib = _lib.load_library()
    _check_2d("w", w, _BF16)
    rows, cols = w.shape
    q = _empty((rows, cols), torch.uint8, w.device, stream)
    q_t = _empty((cols, rows), torch.uint8, w.device, stream) if transposed else None
    scales = _empty((rows // 128, cols // 128), torch.float32, w.device, stream)
    if tiled:
        st = lib.fp8_quant_weight_128x128_tiled(_ptr(w), rows, cols, w.stride(0), _ptr(q), _ptr(q_t),
                                                _ptr(scales), scales.stride(0), _stream(stream))
        _lib.check("fp8_quant_weight_128x128_tiled", st)
        return q, scales, q_t
    st = lib.fp8_quant_weight_128x128(
        _ptr(w), rows, cols, w.stride(0), _ptr(q), q.stride(0), _ptr(q_t),
        q_t.stride(0) if q_t is not None else 0, _ptr(scales), scales.stride(0), _stream(stream))
    _lib.check("fp8_quant_weight_128x128", st)
    return q, scales, q_t


def block_gemm_noalloc(layout: str, A: torch.Tensor, sA: torch.Tensor, B: torch.Tensor, sB: torch.Tensor,
                       *, out, stream=None):
    """block_gemm through fp8_block_gemm_noalloc: the library allocates
    nothing (its split workspace is a static device array shared by every call
    on the GPU; calls that overlap in time on one GPU race).  `out` is the
    caller's C [M][N] (bfloat16 or float32)."""
    return block_gemm(layout, A, sA, B, sB, out=out, stream=stream, _entry="fp8_block_gemm_noalloc")


def block_gemm(layout: str, A: torch.Tensor, sA: torch.Tensor, B: torch.Tensor, sB: torch.Tensor,
               *, out_dtype=torch.bfloat16, out=None, stream=None, _entry="fp8_block_gemm"):
    """Block-scaled FP8 GEMM.

    fprop: A [M][K], sA [K/128][>=M], B [N][K], sB [N/128][>=K/128]
    dgrad: A [M][K], sA [K/128][>=M], B [K][N] (forward W_q), sB [K/128][>=N/128]
    dgrad_t: A [M][K], sA [K/128][>=M], B [N][K] (W_q^T, the q_t of the weight
             quantizer), sB [K/128][>=N/128] (the forward block-scale table)
    wgrad: A [M][K], sA [K/128][>=M], B [N][K], sB [K/128][>=N]
    fprop_tiled / dgrad_t_tiled / wgrad_tiled: as fprop / dgrad_t / wgrad with
             B holding the operand-tiled bytes (quant_weight_128x128(...,
             tiled=True); for wgrad quant_act_1x128(x, "col_tiled") or
             quant_act_dual(x, tiled=True))
    Returns C [M][N] in out_dtype (bfloat16 or float32).
    """
    lib = _lib.load_library()
    for n, t in (("A", A), ("B", B)):
        _check_2d(n, t, (torch.uint8, torch.float8_e4m3fn))
    _check_2d("sA", sA, (torch.float32,))
    _check_2d("sB", sB, (torch.float32,))
    M, K = A.shape
    N = B.shape[1] if layout == "dgrad" else B.shape[0]
    if out is None:
        out = _empty((M, N), out_dtype, A.device, stream)
    code = _lib.OUT_FP32 if out.dtype == torch.float32 else _lib.OUT_BF16
    st = getattr(lib, _entry)(
        _lib.LAYOUT[layout], M, N, K, _ptr(A), A.stride(0), _ptr(sA), sA.stride(0),
        _ptr(B), B.stride(0), _ptr(sB), sB.stride(0), _ptr(out), code, out.stride(0),
        _stream(stream))
    _lib.check(_entry, st)
    return out


def block_gemm_fused_quant(x: torch.Tensor, W: torch.Tensor, sW: torch.Tensor, *, out_dtype=torch.bfloat16,
                           with_codes: bool = False, out=None, stream=None):
    """Fprop with the 1x128 quantization of X fused into the GEMM.

    x: bfloat16 [M][K]; W: codes [N][K] (row-major); sW [N/128][>=K/128].
    Returns C [M][N] (out_dtype), equal bit for bit to
    block_gemm("fprop", *quant_act_1x128(x, "row")[:2], W, sW); with
    with_codes=True returns (C, codes [M][K], scales [K/128][M_pad]) as the
    kernel formed them.
    """
    lib = _lib.load_library()
    _check_2d("x", x, _BF16)
    _check_2d("W", W, (torch.uint8, torch.float8_e4m3fn))
    _check_2d("sW", sW, (torch.float32,))
    M, K = x.shape
    N = W.shape[0]
    if out is None:
        out = _empty((M, N), out_dtype, x.device, stream)
    code = _lib.OUT_FP32 if out.dtype == torch.float32 else _lib.OUT_BF16
    q = s = None
    if with_codes:
        q = _empty((M, K), torch.uint8, x.device, stream)
        s = _empty((K // 128, round_up(M, 4)), torch.float32, x.device, stream)
    st = lib.fp8_block_gemm_fused_quant(
        M, N, K, _ptr(x), x.stride(0), _ptr(W), W.stride(0), _ptr(sW), sW.stride(0), _ptr(out), code,
        out.stride(0), _ptr(q) if q is not None else None, q.stride(0) if q is not None else 0,
        _ptr(s) if s is not None else None, s.stride(0) if s is not None else 0, _stream(stream))
    _lib.check("fp8_block_gemm_fused_quant", st)
    return (out, q, s) if with_codes else out


def block_gemm_grouped(offsets: torch.Tensor, A: torch.Tensor, sA: torch.Tensor, B: torch.Tensor,
                       sB: torch.Tensor, *, tiled: bool = False, out_dtype=torch.bfloat16, out=None,
                       stream=None):
    """Grouped per-expert Fprop in one launch.

    offsets: int32 device [G+1]; A [total_M][K]; sA [K/128][>=total_M];
    B [G][N][K] (operand-tiled bytes per expert if tiled); sB [G][N/128][K/128].
    Returns C [total_M][N].
    """
    lib = _lib.load_library()
    _check_2d("A", A, (torch.uint8, torch.float8_e4m3fn))
    _check_2d("sA", sA, (torch.float32,))
    if B.dim() != 3 or not B.is_contiguous() or sB.dim() != 3 or not sB.is_contiguous():
        raise ValueError("B must be contiguous [G][N][K] and sB contiguous [G][N/128][K/128]")
    if offsets.dtype != torch.int32 or not offsets.is_cuda:
        raise TypeError("offsets must be an int32 device tensor")
    G, N, K = B.shape
    total_M = A.shape[0]
    if out is None:
        out = _empty((total_M, N), out_dtype, A.device, stream)
    code = _lib.OUT_FP32 if out.dtype == torch.float32 else _lib.OUT_BF16
    if tiled:
        st = lib.fp8_block_gemm_grouped_tiled(
            G, _ptr(offsets), total_M, N, K, _ptr(A), A.stride(0), _ptr(sA), sA.stride(0),
            _ptr(B), _ptr(sB), _ptr(out), code, out.stride(0), _stream(stream))
        _lib.check("fp8_block_gemm_grouped_tiled", st)
        return out
    st = lib.fp8_block_gemm_grouped(
        G, _ptr(offsets), total_M, N, K, _ptr(A), A.stride(0), _ptr(sA), sA.stride(0),
        _ptr(B), B.stride(1), _ptr(sB), _ptr(out), code, out.stride(0), _stream(stream))
    _lib.check("fp8_block_gemm_grouped", st)
    return out


def amax_history_update(hist: torch.Tensor, amax: torch.Tensor, *, decay: float = 0.9,
                        init: bool = False, scales_out=None, stream=None):
    """In-place h <- decay * h + (1 - decay) * amax (or h <- amax when init)."""
    lib = _lib.load_library()
    for n, t in (("hist", hist), ("amax", amax)):
        if t.dtype != torch.float32 or not t.is_contiguous() or not t.is_cuda:
            raise ValueError(f"{n}: contiguous float32 device tensor required")
    st = lib.fp8_amax_history_update(_ptr(hist), _ptr(amax), hist.numel(), float(decay),
                                     1 if init else 0, _ptr(scales_out), _stream(stream))
    _lib.check("fp8_amax_history_update", st)
    return hist


def cast_e4m3(x: torch.Tensor, *, out=None, stream=None):
    """Saturating round-to-nearest-even FP32 -> E4M3 codes (uint8)."""
    lib = _lib.load_library()
    if x.dtype != torch.float32 or not x.is_contiguous() or not x.is_cuda:
        raise ValueError("x: contiguous float32 device tensor required")
    if out is None:
        out = _empty(x.shape, torch.uint8, x.device, stream)
    st = lib.fp8_cast_e4m3(_ptr(x), x.numel(), _ptr(out), _stream(stream))
    _lib.check("fp8_cast_e4m3", st)
    return out


def message_bytes(H: int) -> int:
    """Bytes of one token message: H codes + H/128 FP32 scales."""
    return H + H // 32


def pack_tokens(x: torch.Tensor, src_rows=None, *, T=None, stride=None, out=None, stream=None):
    """Quantize tokens x [rows][H] BF16 into messages uint8 [T][stride].

    src_rows: optional int32 device tensor [T]; message t carries row
    src_rows[t] (dispatch order).  Default: every row in order.
    stride defaults to round_up(H + H/32, 16).
    """
    lib = _lib.load_library()
    _check_2d("x", x, _BF16)
    rows, H = x.shape
    if src_rows is not None:
        if src_rows.dtype != torch.int32 or src_rows.dim() != 1 or not src_rows.is_contiguous():
            raise ValueError("src_rows: contiguous 1-D int32 device tensor required")
        T = src_rows.numel()
    elif T is None:
        T = rows
    stride = round_up(message_bytes(H), 16) if stride is None else stride
    if out is None:
        out = _empty((T, stride), torch.uint8, x.device, stream)
    st = lib.fp8_pack_tokens(_ptr(x), rows, H, x.stride(0), _ptr(src_rows), T, _ptr(out),
                             out.stride(0), _stream(stream))
    _lib.check("fp8_pack_tokens", st)
    return out


def unpack_tokens(msg: torch.Tensor, H: int, *, stream=None):
    """Messages [T][stride] -> (q [T][H] uint8, scales [H/128][round_up(T, 4)] float32),
    the operand layout of quant_act_1x128(..., "row")."""
    lib = _lib.load_library()
    _check_2d("msg", msg, (torch.uint8,))
    T = msg.shape[0]
    q = _empty((T, H), torch.uint8, msg.device, stream)
    s = _empty((H // 128, round_up(T, 4)), torch.float32, msg.device, stream)
    st = lib.fp8_unpack_tokens(_ptr(msg), T, H, msg.stride(0), _ptr(q), q.stride(0), _ptr(s),
                               s.stride(0), _stream(stream))
    _lib.check("fp8_unpack_tokens", st)
    return q, s


def dequant_tokens(msg: torch.Tensor, H: int, *, stream=None):
    """Messages [T][stride] -> BF16 [T][H]: decode(q) * s rounded once to BF16."""
    lib = _lib.load_library()
    _check_2d("msg", msg, (torch.uint8,))
    T = msg.shape[0]
    y = _empty((T, H), torch.bfloat16, msg.device, stream)
    st = lib.fp8_dequant_tokens(_ptr(msg), T, H, msg.stride(0), _ptr(y), y.stride(0), _stream(stream))
    _lib.check("fp8_dequant_tokens", st)
    return y


def gemm_promotion(A: torch.Tensor, B: torch.Tensor, promote_k: int, *, stream=None):
    """C [M][N] FP32 = A [M][K] . B [N][K]^T over E4M3 codes (unit scales), with
    the matrix unit's accumulator promoted to FP32 every promote_k values of K
    (32, 64 or a multiple of 128; >= K: one accumulator chain)."""
    lib = _lib.load_library()
    _check_2d("A", A, (torch.uint8,))
    _check_2d("B", B, (torch.uint8,))
    M, K = A.shape
    N = B.shape[0]
    if B.shape[1] != K:
        raise ValueError(f"A {tuple(A.shape)} and B {tuple(B.shape)}: K differs")
    C = _empty((M, N), torch.float32, A.device, stream)
    st = lib.fp8_gemm_promotion(_ptr(A), M, K, A.stride(0), _ptr(B), N, B.stride(0), promote_k,
                                _ptr(C), C.stride(0), _stream(stream))
    _lib.check("fp8_gemm_promotion", st)
    return C


PROBE_MFMA_MODES = {"plain": 0, "scaled": 1, "fold": 2}


def probe_mfma(codes: torch.Tensor, workgroups: int, iters: int, mode: str = "plain", *, stream=None):
    """Measurement aid: `workgroups` x 4 waves each run 8 * iters independent
    FP8 MFMAs (65,536 FLOP each) on operands taken from `codes` (4096 uint8
    E4M3 codes: A from bytes 32 l.., B from 2048 + 32 l.. for lane l), with no
    memory traffic.  mode: "plain" (the GEMMs' MFMA), "scaled" (its
    block-scaled encoding, scales 2^0) or "fold" (plain MFMAs each followed by
    the 4 FP32 FMAs of the GEMMs' per-block fold).  Returns the per-lane
    checksums [workgroups * 256] float32."""
    lib = _lib.load_library()
    if codes.dtype != torch.uint8 or codes.numel() < 4096 or not codes.is_contiguous():
        raise ValueError("codes: a contiguous uint8 tensor of at least 4096 elements")
    if mode not in PROBE_MFMA_MODES:
        raise ValueError(f"mode: one of {sorted(PROBE_MFMA_MODES)}")
    out = _empty(workgroups * 256, torch.float32, codes.device, stream)
    st = lib.fp8_probe_mfma(workgroups, iters, PROBE_MFMA_MODES[mode], _ptr(codes), _ptr(out), _stream(stream))
    _lib.check("fp8_probe_mfma", st)
    return out


def probe_recip_online(s: torch.Tensor, *, stream=None):
    """Verification aid: the quantizers' reciprocal of each online scale in s
    (float32 device tensor); returns r of the same shape."""
    lib = _lib.load_library()
    if s.dtype != torch.float32 or not s.is_contiguous():
        raise ValueError("s: a contiguous float32 tensor")
    r = _empty_as(s, stream)
    st = lib.fp8_probe_recip_online(_ptr(s), _ptr(r), s.numel(), _stream(stream))
    _lib.check("fp8_probe_recip_online", st)
    return r


def probe_gemm_split(tiles: int, K: int, *, stream=None):
    """Measurement aid: (split_tiles, pieces) - how the persistent GEMM kernel
    schedules `tiles` output tiles of 128 x 256 with K-dimension K on `stream`:
    the number of leftover tiles cut along K and the pieces per such tile
    (0, 1: whole tiles only)."""
    lib = _lib.load_library()
    n = ctypes.c_int64(0)
    k = ctypes.c_int32(0)
    st = lib.fp8_probe_gemm_split(tiles, K, _stream(stream), ctypes.byref(n), ctypes.byref(k))
    _lib.check("fp8_probe_gemm_split", st)
    return n.value, k.value


def quant_act_tiles(x: torch.Tensor, tile: int = 128, rank: int = 1, *, sat_count=None, stream=None):
    """1 x tile quantization of x [rows][cols] BF16 with the clip value at the
    rank-th largest |x| of each tile (rank 1: the max).  Returns
    (q [rows][cols] uint8, scales [cols/tile][round_up(rows, 4)] float32).
    sat_count: optional one-element int32/uint32 device tensor, incremented."""
    lib = _lib.load_library()
    _check_2d("x", x, _BF16)
    rows, cols = x.shape
    q = _empty((rows, cols), torch.uint8, x.device, stream)
    s = _empty((cols // tile, round_up(rows, 4)), torch.float32, x.device, stream)
    st = lib.fp8_quant_act_tiles(_ptr(x), rows, cols, x.stride(0), tile, rank, _ptr(q), q.stride(0),
                                 _ptr(s), s.stride(0), _ptr(sat_count), _stream(stream))
    _lib.check("fp8_quant_act_tiles", st)
    return q, s


_FLOATS = (torch.bfloat16, torch.float32)
_FP32 = (torch.float32,)
_CODES = (torch.uint8, torch.float8_e4m3fn)


def _float_type(dtype):
    if dtype not in _FLOATS:
        raise TypeError(f"out_dtype: {dtype} not in {_FLOATS}")
    return dtype


def _is_fp32(t: torch.Tensor) -> int:
    return _lib.OUT_FP32 if t.dtype == torch.float32 else _lib.OUT_BF16


def _check_vec(name, t, n, dtypes):
    if t is None:
        return
    if t.dtype not in dtypes or t.shape != (n,) or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name}: a contiguous device vector of {n} elements of {dtypes} is required, got "
                         f"{t.dtype} {tuple(t.shape)}")


def _norm_affine(weight, bias, cols):
    _check_vec("weight", weight, cols, _FLOATS)
    _check_vec("bias", bias, cols, _FLOATS)
    t = weight if weight is not None else bias
    if t is None:
        return _lib.OUT_BF16
    if bias is not None and bias.dtype != t.dtype:
        raise TypeError(f"weight is {weight.dtype} and bias {bias.dtype}: one type is required")
    return _is_fp32(t)


def _same_device(dev, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name}: on {t.device}, the input is on {dev}")


def _row_statistics(rows, cols, device, stream):
    """Memory for a norm's mean and rstd.  Rows without columns have neither:
    NaN here, as the library writes nothing then."""
    mean = _empty(rows, torch.float32, device, stream)
    rstd = _empty_as(mean, stream)
    if cols == 0:
        with torch.cuda.stream(stream):
            mean.fill_(float("nan"))
            rstd.fill_(float("nan"))
    return mean, rstd


def layer_norm(x: torch.Tensor, weight=None, bias=None, *, eps: float = 1e-5, return_stats: bool = False,
               out=None, stream=None):
    """Layer norm over the rows of x [rows][cols] (bfloat16 or float32).

    weight, bias: optional [cols] vectors of one type (bfloat16 or float32).
    Returns y in x's type, or (y, mean, rstd) with the float32 row statistics
    that layer_norm_backward takes (NaN for rows without columns).
    """
    lib = _lib.load_library()
    _check_2d("x", x, _FLOATS)
    rows, cols = x.shape
    wt = _norm_affine(weight, bias, cols)
    _same_device(x.device, weight=weight, bias=bias, out=out)
    if out is None:
        out = _empty_as(x, stream)
    else:
        _check_2d("out", out, (x.dtype,))
        if out.shape != x.shape:
            raise ValueError(f"out: expected {tuple(x.shape)}, got {tuple(out.shape)}")
    mean, rstd = _row_statistics(rows, cols, x.device, stream) if return_stats else (None, None)
    st = lib.fp8_layer_norm(_ptr(x), rows, cols, x.stride(0), _is_fp32(x), _ptr(weight), _ptr(bias), wt, eps,
                            _ptr(out), out.stride(0), _ptr(mean), _ptr(rstd), None, 0, None, 0, _stream(stream))
    _lib.check("fp8_layer_norm", st)
    return (out, mean, rstd) if return_stats else out


def layer_norm_quant(x: torch.Tensor, weight=None, bias=None, *, eps: float = 1e-5, return_y: bool = False,
                     return_stats: bool = False, stream=None):
    """Layer norm of x [rows][cols] with the 1x128 quantization of the result
    fused in: (q [rows][cols] uint8, s [cols/128][round_up(rows, 4)] float32),
    the operand layout of quant_act_1x128(..., "row"), quantized from the FP32
    result.  return_y appends y (x's type); return_stats appends mean, rstd.
    """
    lib = _lib.load_library()
    _check_2d("x", x, _FLOATS)
    rows, cols = x.shape
    wt = _norm_affine(weight, bias, cols)
    _same_device(x.device, weight=weight, bias=bias)
    q = _empty((rows, cols), torch.uint8, x.device, stream)
    s = _empty((cols // 128, round_up(rows, 4)), torch.float32, x.device, stream)
    y = _empty((rows, cols), x.dtype, x.device, stream) if return_y else None
    mean, rstd = _row_statistics(rows, cols, x.device, stream) if return_stats else (None, None)
    st = lib.fp8_layer_norm(_ptr(x), rows, cols, x.stride(0), _is_fp32(x), _ptr(weight), _ptr(bias), wt, eps,
                            _ptr(y), cols, _ptr(mean), _ptr(rstd), _ptr(q), cols, _ptr(s), s.stride(0),
                            _stream(stream))
    _lib.check("fp8_layer_norm", st)
    return (q, s) + ((y,) if return_y else ()) + ((mean, rstd) if return_stats else ())


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor, weight=None, *,
                        stream=None):
    """Gradients of layer_norm: (dx in x's type, dweight, dbias float32 [cols]).

    dy and x: [rows][cols] of one type; mean, rstd: the statistics that
    layer_norm(..., return_stats=True) returned; weight: as in the forward.
    """
    lib = _lib.load_library()
    _check_2d("x", x, _FLOATS)
    _check_2d("dy", dy, (x.dtype,))
    if dy.shape != x.shape:
        raise ValueError(f"dy {tuple(dy.shape)} and x {tuple(x.shape)} differ")
    rows, cols = x.shape
    wt = _norm_affine(weight, None, cols)
    _check_vec("mean", mean, rows, (torch.float32,))
    _check_vec("rstd", rstd, rows, (torch.float32,))
    _same_device(x.device, dy=dy, mean=mean, rstd=rstd, weight=weight)
    dx = _empty_as(x, stream)
    dweight = _empty(cols, torch.float32, x.device, stream)
    dbias = _empty_as(dweight, stream)
    nbytes = lib.fp8_layer_norm_backward_workspace(rows, cols)
    ws = _workspace(nbytes, x.device, stream)
    st = lib.fp8_layer_norm_backward(_ptr(dy), dy.stride(0), _ptr(x), x.stride(0), rows, cols, _is_fp32(x),
                                     _ptr(mean), _ptr(rstd), _ptr(weight), wt, _ptr(dx), dx.stride(0),
                                     _ptr(dweight), _ptr(dbias), _ptr(ws), nbytes, _stream(stream))
    _lib.check("fp8_layer_norm_backward", st)
    return dx, dweight, dbias


def _check_codes(name, t, shape):
    if t.dtype not in (torch.uint8, torch.float8_e4m3fn) or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name}: contiguous E4M3 codes {shape} required, got {t.dtype} {tuple(t.shape)}")


def _check_scales(name, t, shape):
    if t.dtype != torch.float32 or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name}: contiguous float32 {shape} required, got {t.dtype} {tuple(t.shape)}")


def moe_few_tokens(x: torch.Tensor, router: torch.Tensor, w13: torch.Tensor, s13: torch.Tensor, w2: torch.Tensor,
                   s2: torch.Tensor, *, top_k: int, gate: str = "softmax", bias=None, normalize: bool = True,
                   scale: float = 1.0, first_expert: int = 0, return_routing: bool = False,
                   out_dtype=torch.bfloat16, out=None, stream=None):
    """A whole mixture-of-experts layer for up to 64 tokens x [T][H] bfloat16.

    router: bfloat16 [E][H]; gate: "softmax" or "sigmoid"; bias: optional
    float32 [E] added to the sigmoid scores for the choice only; the chosen
    scores are normalized to sum 1 (normalize) and multiplied by scale.
    w13 [local][2 I][H], w2 [local][H][I]: operand-tiled codes, each expert
    quantized by quant_weight_128x128(..., tiled=True) (w13: gate rows, then
    up rows), with block scales s13 [local][2 I/128][H/128] and s2
    [local][H/128][I/128].  The experts held are first_expert ..
    first_expert + local - 1 of E; the others' contributions are left out.
    Returns y [T][H] in out_dtype, or (y, ids int32 [T][top_k], gates float32
    [T][top_k]) with return_routing.
    """
    lib = _lib.load_library()
    _check_2d("x", x, (torch.bfloat16,))
    _check_2d("router", router, (torch.bfloat16,))
    T, H = x.shape
    E = router.shape[0]
    if router.shape[1] != H or w2.dim() != 3 or gate not in _lib.MOE_GATE:
        raise ValueError(f"x {tuple(x.shape)}, router {tuple(router.shape)}, w2 {tuple(w2.shape)}, gate {gate!r}")
    local, _, I = w2.shape
    _check_codes("w13", w13, (local, 2 * I, H))
    _check_codes("w2", w2, (local, H, I))
    _check_scales("s13", s13, (local, 2 * I // 128, H // 128))
    _check_scales("s2", s2, (local, H // 128, I // 128))
    _check_vec("bias", bias, E, (torch.float32,))
    _same_device(x.device, router=router, w13=w13, s13=s13, w2=w2, s2=s2, bias=bias, out=out)
    if out is None:
        out = _empty((T, H), _float_type(out_dtype), x.device, stream)
    else:
        _check_2d("out", out, _FLOATS)
        if out.shape != x.shape:
            raise ValueError(f"out: expected {tuple(x.shape)}, got {tuple(out.shape)}")
    ids = gates = None
    if return_routing:
        ids = _empty((T, top_k), torch.int32, x.device, stream)
        gates = _empty((T, top_k), torch.float32, x.device, stream)
    nbytes = lib.fp8_moe_few_tokens_workspace(T, H, I, E, local, top_k)
    ws = _workspace(nbytes, x.device, stream)
    st = lib.fp8_moe_few_tokens(T, H, I, E, first_expert, local, top_k, _ptr(x), x.stride(0), _ptr(router),
                                router.stride(0), _ptr(bias), _lib.MOE_GATE[gate], int(normalize), scale, _ptr(w13),
                                _ptr(s13), _ptr(w2), _ptr(s2), _ptr(out), _is_fp32(out), out.stride(0), _ptr(ids),
                                _ptr(gates), _ptr(ws), nbytes, _stream(stream))
    _lib.check("fp8_moe_few_tokens", st)
    return (out, ids, gates) if return_routing else out


def adapter_linear(x: torch.Tensor, w: torch.Tensor, sw: torch.Tensor, lora_a: torch.Tensor, lora_b: torch.Tensor,
                   ids: torch.Tensor, *, scales=None, out_dtype=torch.bfloat16, out=None, stream=None):
    """A shared FP8 projection with a low-rank adapter of its own per token:
    y[t] = W_q . quant_1x128(x[t]) + scales[a] * lora_b[a] . (lora_a[a] . x[t])
    with a = ids[t] (negative: no adapter).

    x: bfloat16 [T][K]; w [N][K]: operand-tiled codes of
    quant_weight_128x128(..., tiled=True), sw its block scales; lora_a bfloat16
    [n][rank][K], lora_b bfloat16 [n][N][rank] (rank % 8 == 0, <= 128); ids int32
    [T]; scales: optional float32 [n].  Returns y [T][N] in out_dtype.
    """
    lib = _lib.load_library()
    _check_2d("x", x, (torch.bfloat16,))
    _check_2d("sw", sw, (torch.float32,))
    T, K = x.shape
    if lora_a.dim() != 3 or lora_b.dim() != 3 or w.dim() != 2:
        raise ValueError("w, lora_a, lora_b: expected [N][K], [n][rank][K], [n][N][rank]")
    N = w.shape[0]
    n, r, _ = lora_a.shape
    _check_codes("w", w, (N, K))
    if sw.shape[0] < N // 128 or sw.shape[1] < K // 128:
        raise ValueError(f"sw: expected at least {(N // 128, K // 128)}, got {tuple(sw.shape)}")
    for name, t, shape in (("lora_a", lora_a, (n, r, K)), ("lora_b", lora_b, (n, N, r))):
        if t.dtype != torch.bfloat16 or tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"{name}: contiguous bfloat16 {shape} required, got {t.dtype} {tuple(t.shape)}")
    _check_vec("ids", ids, T, (torch.int32,))
    _check_vec("scales", scales, n, (torch.float32,))
    _same_device(x.device, w=w, sw=sw, lora_a=lora_a, lora_b=lora_b, ids=ids, scales=scales, out=out)
    if out is None:
        out = _empty((T, N), _float_type(out_dtype), x.device, stream)
    else:
        _check_2d("out", out, _FLOATS)
        if tuple(out.shape) != (T, N):
            raise ValueError(f"out: expected {(T, N)}, got {tuple(out.shape)}")
    nbytes = lib.fp8_adapter_linear_workspace(T, N, K, r, n)
    ws = _workspace(nbytes, x.device, stream)
    st = lib.fp8_adapter_linear(T, N, K, r, n, _ptr(x), x.stride(0), _ptr(w), _ptr(sw), sw.stride(0), _ptr(lora_a),
                                _ptr(lora_b), _ptr(ids), _ptr(scales), _ptr(out), _is_fp32(out), out.stride(0),
                                _ptr(ws), nbytes, _stream(stream))
    _lib.check("fp8_adapter_linear", st)
    return out


def _on_current_device(name, t):
    """Launches go to the current device: a tensor of another one is refused."""
    index = t.get_device()
    if index >= 0 and index != torch._C._cuda_getDevice():      # a tensor there: the runtime is up
        raise ValueError(f"{name}: on {t.device}, the current device is cuda:{torch.cuda.current_device()}")


def _activation(name):
    if name not in _lib.ACTIVATION:
        raise ValueError(f"activation: {name!r} not in {sorted(_lib.ACTIVATION)}")
    return _lib.ACTIVATION[name]


# what the library answers for these sizes, asked for once (a call into it takes
# half a microsecond)
@functools.lru_cache(maxsize=4096)
def _gated_workspace(M, I, K, h_type, codes):
    return _lib.load_library().fp8_block_gemm_gated_workspace(M, I, K, h_type, codes)


@functools.lru_cache(maxsize=4096)
def _heads_workspace(T, heads_q, heads_k, dim):
    return _lib.load_library().fp8_head_norm_rotary_backward_workspace(T, heads_q, heads_k, dim)


def _rows(name, t, dtypes, rows, cols, dev):
    """t has at least [rows][cols] of these types, row-major, on this device; its row stride."""
    shape, strides = t.shape, t.stride()
    if len(shape) != 2 or strides[1] != 1 or shape[0] < rows or shape[1] < cols:
        raise ValueError(f"{name}: expected row-major, at least {(rows, cols)}, got {tuple(shape)} strides {strides}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, expected cuda:{dev}")
    return strides[0]


def _made(like, shape, dtype, stream):
    """An uninitialized tensor on like's device (the short call on the current stream)."""
    return like.new_empty(shape, dtype=dtype) if stream is None else _empty(shape, dtype, like.device, stream)


def _scratch(like, nbytes, stream):
    """_workspace on like's device (the short call on the current stream)."""
    return like.new_empty(max(nbytes, 0), dtype=torch.uint8) if stream is None else _workspace(nbytes, like.device, stream)


def _gated(A, sA, w13, s13, activation, quant, return_gate_up, out_dtype, out, stream):
    lib = _lib.load_library()
    act = _activation(activation)
    _check_2d("A", A, _CODES)
    _on_current_device("A", A)
    dev = A.get_device()
    M, K = A.shape
    rows = w13.shape[0] if w13.dim() == 2 else 1
    if rows % 2 != 0:
        raise ValueError(f"w13: expected [2 I][K], got {tuple(w13.shape)}")
    I = rows // 2
    _check_codes("w13", w13, (rows, K))
    if w13.get_device() != dev:
        raise ValueError(f"w13: on {w13.device}, the input is on {A.device}")
    ld_sa = _rows("sA", sA, _FP32, K // 128, M, dev)
    ld_s13 = _rows("s13", s13, _FP32, rows // 128, K // 128, dev)
    q = s = gate_up = ws = None
    ldh = ld_s = h_type = 0
    if quant:
        ld_s = round_up(M, 4)
        q = _made(A, (M, I), torch.uint8, stream)
        s = _made(A, (I // 128, ld_s), torch.float32, stream)
    else:
        if out is None:
            out = _made(A, (M, I), _float_type(out_dtype), stream)
            ldh = I
        else:
            ldh = _rows("out", out, _FLOATS, M, I, dev)
            if out.shape != (M, I):
                raise ValueError(f"out: expected {(M, I)}, got {tuple(out.shape)}")
        h_type = _is_fp32(out)
    if return_gate_up:
        gate_up = _made(A, (M, rows), torch.bfloat16, stream)
    nbytes = _gated_workspace(M, I, K, h_type, quant)
    if nbytes != 0:
        ws = _scratch(A, nbytes, stream)
    st = lib.fp8_block_gemm_gated(
        M, I, K, A.data_ptr(), A.stride(0), sA.data_ptr(), ld_sa, w13.data_ptr(), s13.data_ptr(), ld_s13, act,
        _ptr(out), h_type, ldh, _ptr(gate_up), rows, _ptr(q), I, _ptr(s), ld_s, _ptr(ws), nbytes, _stream(stream))
    if st != 0:
        _lib.check("fp8_block_gemm_gated", st)
    return out, q, s, gate_up


def block_gemm_gated(A: torch.Tensor, sA: torch.Tensor, w13: torch.Tensor, s13: torch.Tensor, *,
                     activation: str = "silu", return_gate_up: bool = False, out_dtype=torch.bfloat16, out=None,
                     stream=None):
    """The gated feed-forward product on FP8 codes: h = act(A W1^T) * (A W3^T).

    A [M][K] codes, sA [K/128][>=M] (quant_act_1x128 or layer_norm_quant); w13
    [2 I][K]: operand-tiled codes of quant_weight_128x128(..., tiled=True) of the
    I rows of W1 and then the I rows of W3, s13 [2 I/128][>=K/128] their block
    scales.  activation: "silu" or "gelu" (tanh form).  Returns h [M][I] in
    out_dtype (bfloat16 or float32), or with return_gate_up (h, gate_up): the two
    projections in bfloat16 [M][2 I], which gated_backward_quant takes.  A call repeats
    itself bit for bit; a row moved within a batch of more than 64 may differ in FP32's last
    bits, as the order of its sums follows its place.
    """
    h, _, _, gate_up = _gated(A, sA, w13, s13, activation, False, return_gate_up, out_dtype, out, stream)
    return (h, gate_up) if return_gate_up else h


def block_gemm_gated_quant(A: torch.Tensor, sA: torch.Tensor, w13: torch.Tensor, s13: torch.Tensor, *,
                           activation: str = "silu", return_gate_up: bool = False, stream=None):
    """block_gemm_gated with the 1x128 quantization of h in its epilogue, from the
    FP32 values: (q [M][I] uint8, s [I/128][round_up(M, 4)] float32), the operand of
    the down product; return_gate_up appends gate_up."""
    _, q, s, gate_up = _gated(A, sA, w13, s13, activation, True, return_gate_up, None, None, stream)
    return (q, s, gate_up) if return_gate_up else (q, s)


def _gated_backward(dh, gate_up, activation, stream, d=None, q=None, s=None, qt=None, st=None, ht=None, sht=None):
    T, I = dh.shape
    status = _lib.load_library().fp8_gated_backward(
        T, I, dh.data_ptr(), dh.stride(0), gate_up.data_ptr(), gate_up.stride(0), _activation(activation), _ptr(d), 2 * I,
        _ptr(q), 2 * I, _ptr(s), round_up(T, 4), _ptr(qt), round_up(T, 128), _ptr(st), 2 * I, _ptr(ht), _ptr(sht), I,
        _stream(stream))
    if status != 0:
        _lib.check("fp8_gated_backward", status)


def _check_gated_backward(dh, gate_up):
    _check_2d("dh", dh, (torch.bfloat16,))
    _on_current_device("dh", dh)
    T, I = dh.shape
    _rows("gate_up", gate_up, (torch.bfloat16,), T, 2 * I, dh.get_device())
    if gate_up.shape != (T, 2 * I):
        raise ValueError(f"gate_up: expected {(T, 2 * I)}, got {tuple(gate_up.shape)}")
    return T, I


def gated_backward(dh: torch.Tensor, gate_up: torch.Tensor, *, activation: str = "silu", stream=None):
    """Gradient of h = act(a) * u for dh [T][I] bfloat16 and gate_up = [a | u]
    [T][2 I] bfloat16 (I a multiple of 128): [da | du] [T][2 I] bfloat16."""
    T, I = _check_gated_backward(dh, gate_up)
    d = _made(dh, (T, 2 * I), torch.bfloat16, stream)
    _gated_backward(dh, gate_up, activation, stream, d=d)
    return d


def gated_backward_quant(dh: torch.Tensor, gate_up: torch.Tensor, *, activation: str = "silu", return_h: bool = False,
                         stream=None):
    """gated_backward with both orientations of its result's codes in one pass,
    formed from FP32 values: (q [T][2 I] uint8, s [2 I/128][round_up(T, 4)]) of the
    1x128 row tiles for "dgrad_t_tiled", and (qt [2 I][Tp], st [Tp/128][2 I]) of the
    128x1 column tiles, transposed, for the A side of "wgrad_tiled".  Any T; Tp = T
    rounded up to 128, the rows past T counting as zeros (quant_act_cols pads the
    other operand alike).  return_h appends (ht [I][Tp], sht [Tp/128][I]): h's column
    tiles, operand-tiled, for the weight gradient of the down projection."""
    T, I = _check_gated_backward(dh, gate_up)
    Tp = round_up(T, 128)
    q = _made(dh, (T, 2 * I), torch.uint8, stream)
    s = _made(dh, (2 * I // 128, round_up(T, 4)), torch.float32, stream)
    qt = _made(dh, (2 * I, Tp), torch.uint8, stream)
    st = _made(dh, (Tp // 128, 2 * I), torch.float32, stream)
    ht = sht = None
    if return_h:
        ht = _made(dh, (I, Tp), torch.uint8, stream)
        sht = _made(dh, (Tp // 128, I), torch.float32, stream)
    _gated_backward(dh, gate_up, activation, stream, None, q, s, qt, st, ht, sht)
    return (q, s, qt, st, ht, sht) if return_h else (q, s, qt, st)


def quant_act_cols(x: torch.Tensor, *, stream=None):
    """quant_act_1x128(x, "col_tiled") for any number of rows: (q [cols][Tp] uint8,
    operand-tiled, s [Tp/128][cols] float32) with Tp = rows rounded up to 128, the rows
    past the last one counting as zeros.  x: bfloat16 [rows][cols], cols a multiple
    of 128."""
    lib = _lib.load_library()
    _check_2d("x", x, _BF16)
    _on_current_device("x", x)
    rows, cols = x.shape
    Tp = round_up(rows, 128)
    q = _made(x, (cols, Tp), torch.uint8, stream)
    s = _made(x, (Tp // 128, cols), torch.float32, stream)
    st = lib.fp8_quant_act_cols(x.data_ptr(), rows, cols, x.stride(0), q.data_ptr(), s.data_ptr(), cols, _stream(stream))
    if st != 0:
        _lib.check("fp8_quant_act_cols", st)
    return q, s


def _check_heads(name, t, dtype, dev, T, heads, dim):
    """t is [T][heads][dim] (heads None: any number) of this type on this device; its number of heads and strides."""
    shape, strides = t.shape, t.stride()
    if len(shape) != 3 or shape[0] != T or shape[2] != dim or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name}: expected {(T, 'any' if heads is None else heads, dim)}, got {tuple(shape)}")
    if strides[2] != 1 and dim > 1:
        raise ValueError(f"{name}: the channels have to be contiguous, got strides {strides}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, expected cuda:{dev}")
    return shape[1], strides


def _first_heads(q, k):
    """(type, device index, T, dim) that the sets share."""
    t = q if q is not None else k
    if t is None:
        raise ValueError("q, k: at least one is required")
    shape = t.shape
    if len(shape) != 3 or t.dtype not in _FLOATS:
        raise TypeError(f"q, k: expected [tokens][heads][dim] of {_FLOATS}, got {tuple(shape)} {t.dtype}")
    if not t.is_cuda:
        raise ValueError("q, k: must be device tensors")
    _on_current_device("q, k", t)
    return t.dtype, t.get_device(), shape[0], shape[2]


def _head_vector(name, t, n, dev, dtypes):
    if t.dtype not in dtypes or t.shape != (n,) or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name}: a contiguous vector of {n} elements of {dtypes} on cuda:{dev} is required, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")


_POSITION_BYTES = {torch.int64: 8, torch.int32: 4}


def _head_arguments(dev, T, dim, wq, wk, norm, eps, positions, freq, sections, adjacent):
    """The arguments between the sets and the workspace or stream."""
    code = _lib.HEAD_NORM.get(norm, -1)
    if code < 0:
        raise ValueError(f"norm: {norm!r} not in {list(_lib.HEAD_NORM)}")
    wt = _lib.OUT_BF16
    if wq is not None or wk is not None:
        if norm is None:
            raise ValueError("q_weight, k_weight: without a norm there is no weight")
        if wq is not None:
            _head_vector("q_weight", wq, dim, dev, _FLOATS)
            wt = _is_fp32(wq)
        if wk is not None:
            _head_vector("k_weight", wk, dim, dev, _FLOATS if wq is None else (wq.dtype,))
            wt = _is_fp32(wk)
    if freq is None:
        if positions is not None:
            raise ValueError("positions and freq: both or neither")
        return wt, code, eps, 0, None, 8, 1, None, None, 0
    if positions is None:
        raise ValueError("positions and freq: both or neither")
    pairs = freq.numel()
    _head_vector("freq", freq, pairs, dev, (torch.float64,))
    axes, counts = 1, None
    if sections is not None:
        axes = len(sections)
        counts = (ctypes.c_int64 * axes)(*sections)
    shape, nbytes = positions.shape, _POSITION_BYTES.get(positions.dtype)
    if nbytes is None or not positions.is_contiguous() or not (shape == (T, axes) or (axes == 1 and shape == (T,))) or \
            positions.get_device() != dev:
        raise ValueError(f"positions: contiguous int32 or int64 {(T, axes)} on cuda:{dev} required, got {positions.dtype} "
                         f"{tuple(shape)} on {positions.device}")
    return wt, code, eps, 2 * pairs, positions.data_ptr(), nbytes, axes, counts, freq.data_ptr(), 1 if adjacent else 0


def _head_output(name, given, like, index, shape, stream):
    """The set's output (a new contiguous tensor unless one is given) and its strides."""
    if given is not None:
        return given, _check_heads(name, given, like.dtype, index, *shape)[1]
    if stream is None:      # the shorter call
        made = torch.empty_like(like, memory_format=torch.contiguous_format)
    else:
        made = _empty(shape, like.dtype, like.device, stream)
    return made, (shape[1] * shape[2], shape[2])


def head_norm_rotary(q: torch.Tensor, k, positions=None, freq=None, *, q_weight=None, k_weight=None, norm="rms",
                     eps: float = 1e-6, sections=None, adjacent: bool = False, out=None, stream=None):
    """Norm of each query and key head and the rotation by the token's position, in one pass.

    q [tokens][heads][dim], k [tokens][heads_k][dim] (bfloat16 or float32, either may be
    None): contiguous channels, and token by token (as views of a fused projection are)
    or head by head at any strides, nothing twice (expanded tensors are refused).  norm: "rms", "layer" or None; q_weight, k_weight: optional [dim] vectors of one
    type.  freq: float64 device vector of the rotated pairs' frequencies (rot/2 of them;
    rot <= dim, the other channels pass through), usually
    base ** (-2 i / rot); the angle is formed in FP64.  positions: int32 or int64
    [tokens], or [tokens][axes] with sections = how many consecutive pairs follow each
    axis (time, height, width; up to 4).  adjacent: pairs (2 i, 2 i + 1) instead of
    (i, i + rot/2).  positions = freq = None: the norm alone.
    out: optional (q_out, k_out) of q's and k's shapes and type, at strides as q's; the two may
    lie side by side in a token's row.
    Returns (q_out, k_out), None for a set that is None.
    """
    lib = _lib.load_library()
    dtype, dev, T, dim = _first_heads(q, k)
    args = _head_arguments(dev, T, dim, q_weight, k_weight, norm, eps, positions, freq, sections, adjacent)
    made, sets = [None, None], [None, None]
    for i, t, w in ((0, q, q_weight), (1, k, k_weight)):
        if t is None:
            continue
        heads, strides = _check_heads("qk"[i], t, dtype, dev, T, None, dim)
        o, to = _head_output("out", None if out is None else out[i], t, dev, (T, heads, dim), stream)
        made[i] = o
        sets[i] = _lib.Heads(t.data_ptr(), heads, strides[0], strides[1], None if w is None else w.data_ptr(), o.data_ptr(), to[0],
                             to[1])
    st = lib.fp8_head_norm_rotary(T, dim, _lib.OUT_FP32 if dtype == torch.float32 else _lib.OUT_BF16, sets[0], sets[1], *args,
                                  _stream(stream))
    if st != 0:
        _lib.check("fp8_head_norm_rotary", st)
    return made[0], made[1]


def head_norm_rotary_backward(dq: torch.Tensor, dk, q, k, positions=None, freq=None, *, q_weight=None, k_weight=None,
                              norm="rms", eps: float = 1e-6, sections=None, adjacent: bool = False, out=None, stream=None):
    """Gradients of head_norm_rotary, from its inputs: (dq_in, dk_in, dq_weight, dk_weight).

    dq, dk: the gradients of its outputs (of the inputs' type; None with the set); q, k and the
    other arguments as in the forward pass.  With norm=None q and k may be None and
    there are no weight gradients (None); otherwise those are float32 [dim], the
    sums over tokens and heads (also where the weight is None: of ones).  out:
    optional (dq_in, dk_in) tensors.
    """
    lib = _lib.load_library()
    dtype, dev, T, dim = _first_heads(dq, dk)
    args = _head_arguments(dev, T, dim, q_weight, k_weight, norm, eps, positions, freq, sections, adjacent)
    made, sets, grads, count = [None, None], [None, None], [None, None], [0, 0]
    for i, d, x, w in ((0, dq, q, q_weight), (1, dk, k, k_weight)):
        if d is None:
            continue
        name = "qk"[i]
        heads, strides = _check_heads("d" + name, d, dtype, dev, T, None, dim)
        count[i] = heads
        of = strides
        if norm is None:
            x = d
        elif x is None:
            raise ValueError(f"{name}: required with a norm")
        else:
            of = _check_heads(name, x, dtype, dev, T, heads, dim)[1]
            grads[i] = _made(d, (dim,), torch.float32, stream)
        o, to = _head_output("out", None if out is None else out[i], d, dev, (T, heads, dim), stream)
        made[i] = o
        sets[i] = _lib.HeadsGrad(x.data_ptr(), heads, of[0], of[1], None if w is None else w.data_ptr(), d.data_ptr(), strides[0],
                                 strides[1], o.data_ptr(), to[0], to[1], _ptr(grads[i]))
    nbytes, ws = 0 if norm is None else _heads_workspace(T, count[0], count[1], dim), None
    if nbytes != 0:
        ws = _scratch(dq if dq is not None else dk, nbytes, stream)
    st = lib.fp8_head_norm_rotary_backward(T, dim, _lib.OUT_FP32 if dtype == torch.float32 else _lib.OUT_BF16, sets[0], sets[1],
                                           *args, _ptr(ws), nbytes, _stream(stream))
    if st != 0:
        _lib.check("fp8_head_norm_rotary_backward", st)
    return made[0], made[1], grads[0], grads[1]
