"""Thin PyTorch-facing binding of libfp8bs.so (argument marshalling only).

Tensors are used for device memory and the current HIP stream; every step of
the computation runs in the library's kernels.  Names follow the C ABI in
include/fp8bs.h.  Scale arrays are MN-major: [K/128][ld] with
ld = round_up(rows, 4) for 1x128 row tiles.
"""
from __future__ import annotations

import ctypes

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
