"""4-bit operands (NVFP4 and MXFP4): the MXFP4 cast, reading back, and the product.

    q = quantize_mxfp4(x, colwise=True)          # x [M, N]: q.row of x, q.col of x transposed
    y = matmul_fp4(q.row, w.row)                 # x @ weight.T
    t = quantize(x, "2d", swizzled=True)         # the NVFP4 cast: t.row and t.col are operands too

A product contracts the last dimension of both operands, so the three
products of a linear layer y = x w^T take the operands as

    y  = matmul_fp4(x.row,  w.row)               # forward
    dx = matmul_fp4(dy.row, w.col)               # input gradient
    dw = matmul_fp4(dy.col, x.col)               # weight gradient

(``linear`` runs them together).
"""
from __future__ import annotations

import struct

import torch

from . import BF16, COLWISE, FP32, ROW_SCALED, ROWWISE, SWIZZLED
from ._call import call

_DTYPES = {torch.bfloat16: BF16, torch.float32: FP32}
_U8, _F32 = torch.uint8, torch.float32


class FP4Operand:
    """E2M1 codes [rows, cols / 2] (or [batch, rows, cols / 2]; two in a byte, uint8) with a scale byte for each block.

    block 16: NVFP4, E4M3 scales and a float32 amax, [1] or [rows] (of a batch: [1] or [batch]); a value is code *
    scale * (amax / 2688).  block 32: MXFP4, powers of two stored as exponent + 127, no amax.  Scales are compact
    ([rows, cols / block]) or in the cuBLAS 128x4 layout (swizzled); their shape is free.
    """
    __slots__ = ("data", "scale", "amax", "block", "swizzled")

    def __init__(self, data: torch.Tensor, scale: torch.Tensor, amax: torch.Tensor | None = None, block: int = 16,
                 swizzled: bool = False):
        self.data, self.scale, self.amax, self.block, self.swizzled = data, scale, amax, block, swizzled

    def __repr__(self) -> str:
        return f"FP4Operand({tuple(self.data.shape)}, block={self.block}, swizzled={self.swizzled})"


class FP4Tensor:
    """The casts of one tensor: ``row`` of x, ``col`` of x transposed (or None)."""
    __slots__ = ("row", "col")

    def __init__(self, row: FP4Operand | None, col: FP4Operand | None):
        self.row, self.col = row, col


def quantize_mxfp4(x: torch.Tensor, rowwise: bool = True, colwise: bool = False, swizzled: bool = False) -> FP4Tensor:
    """Casts x ([M, N], bfloat16 or float32) to MXFP4: E2M1 codes with a power of two for each 32 elements of a row.
    colwise: also the cast of x transposed, from the same pass over x.  N % 32 == 0; colwise also M % 32 == 0;
    swizzled scales: both multiples of 128."""
    shape = x.shape
    if len(shape) != 2:
        raise ValueError("x must be [M, N]")
    if not x.is_cuda or not x.is_contiguous():
        raise ValueError("tensors passed to libnvfp4 must be contiguous CUDA tensors")
    dtype = _DTYPES.get(x.dtype)
    if dtype is None:
        raise TypeError(f"quantize_mxfp4 takes bfloat16 or float32 input, got {x.dtype}")
    M, N = shape
    if N % 32 or colwise and M % 32:
        raise ValueError(f"blocks of 32 do not divide {tuple(shape)}")
    dev = x.device
    row = col = None
    pointers = [None] * 4
    if rowwise:
        data = torch.empty((M, N // 2), dtype=_U8, device=dev)
        scale = torch.empty(M * (N // 32), dtype=_U8, device=dev)
        row = FP4Operand(data, scale, None, 32, swizzled)
        pointers[:2] = data.data_ptr(), scale.data_ptr()
    if colwise:
        data = torch.empty((N, M // 2), dtype=_U8, device=dev)
        scale = torch.empty(N * (M // 32), dtype=_U8, device=dev)
        col = FP4Operand(data, scale, None, 32, swizzled)
        pointers[2:] = data.data_ptr(), scale.data_ptr()
    call("nvfp4_mxfp4_quantize", dev, x.data_ptr(), dtype, M, N, *pointers,
         (ROWWISE if rowwise else 0) | (COLWISE if colwise else 0) | (SWIZZLED if swizzled else 0))
    return FP4Tensor(row, col)


def _check_operand(name: str, q: FP4Operand, dims: int) -> tuple:
    """(batch, rows, cols) of an operand whose parts fit each other.  (In few steps where all is well: a decoding step
    makes many calls of a few microseconds.)"""
    d, s, amax, block = q.data, q.scale, q.amax, q.block
    shape = d.shape
    if len(shape) != dims:
        raise ValueError(f"{name}: codes with {dims} dimensions, got {tuple(shape)}")
    rows, cols = shape[-2], 2 * shape[-1]
    batch = shape[0] if dims == 3 else 1
    dev = d.get_device()
    if d.dtype is not _U8 or s.dtype is not _U8:
        raise TypeError(f"{name}: uint8 codes and scales, got {d.dtype} and {s.dtype}")
    if dev < 0 or s.get_device() < 0 or not (d.is_contiguous() and s.is_contiguous()):
        raise ValueError("tensors passed to libnvfp4 must be contiguous CUDA tensors")
    if s.get_device() != dev:
        raise ValueError(f"{name}: codes and scales on one device")
    if block != 16 and block != 32:
        raise ValueError(f"{name}: block 16 (NVFP4) or 32 (MXFP4), got {block}")
    if cols % 32:
        raise ValueError(f"{name}: the contracted dimension must be a multiple of 32, got {cols}")
    if s.numel() * block != batch * rows * cols:
        raise ValueError(f"{name}: {s.numel()} scales do not fit codes {tuple(shape)} with block {block}")
    if block == 32:
        if amax is not None:
            raise ValueError(f"{name}: an MXFP4 operand has no amax")
    elif amax is None or amax.dtype is not _F32:
        raise TypeError(f"{name}: an NVFP4 operand needs a float32 amax")
    else:
        n = amax.shape
        if len(n) != 1 or n[0] != 1 and n[0] != (batch if dims == 3 else rows):
            raise ValueError(f"{name}: amax {tuple(n)} does not fit codes {tuple(shape)}")
        if amax.get_device() != dev or not amax.is_contiguous():
            raise ValueError(f"{name}: amax must be contiguous, on the codes' device")
    return batch, rows, cols


_pack = struct.Struct("@PPPIi").pack  # nvfp4_operand


def _struct(q: FP4Operand, rows: int) -> bytes:
    """The operand as the library takes it; an amax for each of `rows` or one for all."""
    amax = q.amax
    if amax is None:
        return _pack(q.data.data_ptr(), q.scale.data_ptr(), 0, SWIZZLED if q.swizzled else 0, 0)
    flags = ROW_SCALED if rows != 1 and amax.shape[0] == rows else 0
    return _pack(q.data.data_ptr(), q.scale.data_ptr(), amax.data_ptr(), flags | SWIZZLED if q.swizzled else flags, 0)


def dequantize_fp4(q: FP4Operand, out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """The values of an operand [rows, cols / 2], [rows, cols] in bfloat16 or float32."""
    _, rows, cols = _check_operand("q", q, 2)
    code = _DTYPES.get(out_dtype)
    if code is None:
        raise TypeError(f"values are bfloat16 or float32, not {out_dtype}")
    dev = q.data.device
    out = torch.empty((rows, cols), dtype=out_dtype, device=dev)
    if q.block == 32:
        call("nvfp4_mxfp4_dequantize", dev, q.data.data_ptr(), q.scale.data_ptr(), rows, cols,
             SWIZZLED if q.swizzled else 0, out.data_ptr(), code)
    else:
        scaled = q.amax.numel() == rows and rows != 1
        call("nvfp4_dequantize", dev, q.data.data_ptr(), q.scale.data_ptr(), q.amax.data_ptr(), rows, cols,
             (SWIZZLED if q.swizzled else 0) | (ROW_SCALED if scaled else 0), out.data_ptr(), code)
    return out


def matmul_fp4(a: FP4Operand, b: FP4Operand, out_dtype: torch.dtype = torch.bfloat16,
               out: torch.Tensor | None = None) -> torch.Tensor:
    """a [M, K] times b [N, K] transposed: [M, N] in bfloat16 or float32.

    Both NVFP4 or both MXFP4, scales compact or swizzled, each its own; an amax for each row (the row-scaled cast) or
    one for all.  Summed in FP32 by the tensor cores, rounded once.  K % 32 == 0."""
    _, M, K = _check_operand("a", a, 2)
    _, N, Kb = _check_operand("b", b, 2)
    if K != Kb:
        raise ValueError(f"the contracted dimensions of a ({K}) and b ({Kb}) differ")
    if a.block != b.block:
        raise ValueError("a and b must be of one format")
    dev = a.data.device
    if b.data.get_device() != dev.index:
        raise ValueError("a and b on one device")
    if out is None:
        code = _DTYPES.get(out_dtype)
        if code is not None:
            out = torch.empty((M, N), dtype=out_dtype, device=dev)
    else:
        if out.shape != (M, N) or out.device != dev or not out.is_contiguous():
            raise ValueError(f"out must be a contiguous {(M, N)} tensor on {dev}")
        out_dtype = out.dtype
        code = _DTYPES.get(out_dtype)
    if code is None:
        raise TypeError(f"products are bfloat16 or float32, not {out_dtype}")
    call("nvfp4_fp4_matmul", dev, _struct(a, M), _struct(b, N), a.block, M, N, K, out.data_ptr(), code)
    return out
