"""E4M3 operands with one FP32 scale for each block of 128, and their product.

    q = quantize_fp8(x, colwise=True)            # x [M, N]: q.row of x, q.col of x transposed
    w = quantize_fp8(weight, block_rows=128)     # 128 x 128 blocks
    y = matmul_fp8(q.row, w.row)                 # x @ weight.T

A product contracts the last dimension of both operands, so the three
products of a linear layer y = x w^T take the operands as

    y  = matmul_fp8(x.row,  w.row)               # forward
    dx = matmul_fp8(dy.row, w.col)               # input gradient
    dw = matmul_fp8(dy.col, x.col)               # weight gradient

and by expert, with the member offsets of a ``TokenPlan``, the same through
``matmul_fp8_grouped`` and ``matmul_fp8_grouped_wgrad``.
"""
from __future__ import annotations

import torch

from . import BF16, COLWISE, FP32, ROWWISE
from ._call import call

BLOCK = 128
CODES = torch.float8_e4m3fn


class FP8Operand:
    """E4M3 codes [rows, cols] (or [batch, rows, cols]) and FP32 scales.

    block_rows 1: a scale covers 128 consecutive elements of one row; scale
    [.., ceil(cols/128), rows].  block_rows 128: a 128 x 128 tile; scale
    [.., ceil(rows/128), ceil(cols/128)].
    """
    __slots__ = ("data", "scale", "block_rows")

    def __init__(self, data: torch.Tensor, scale: torch.Tensor, block_rows: int = 1):
        self.data, self.scale, self.block_rows = data, scale, block_rows

    def __repr__(self) -> str:
        return f"FP8Operand({tuple(self.data.shape)}, block_rows={self.block_rows})"

    def dequantize(self) -> torch.Tensor:
        """The values the codes stand for, in FP32 (plain torch; for inspection)."""
        rows, cols = self.data.shape[-2:]
        s = self.scale.transpose(-1, -2) if self.block_rows == 1 else \
            self.scale.repeat_interleave(BLOCK, -2)[..., :rows, :]
        return self.data.float() * s.repeat_interleave(BLOCK, -1)[..., :cols]


class FP8Tensor:
    """The casts of one tensor: ``row`` of x, ``col`` of x transposed (or None)."""
    __slots__ = ("row", "col")

    def __init__(self, row: FP8Operand | None, col: FP8Operand | None):
        self.row, self.col = row, col


def _blocks(n: int) -> int:
    return -(-n // BLOCK)


def _scale_shape(lead: tuple, rows: int, cols: int, block_rows: int) -> tuple:
    return lead + ((_blocks(cols), rows) if block_rows == 1 else (_blocks(rows), _blocks(cols)))


_DTYPES = {torch.bfloat16: BF16, torch.float32: FP32}


def quantize_fp8(x: torch.Tensor, block_rows: int = 1, rowwise: bool = True, colwise: bool = False) -> FP8Tensor:
    """Casts x ([M, N], or a batch [B, M, N] of matrices; bfloat16 or float32)
    to E4M3 with a scale for each block of 128 elements of a row (block_rows 1)
    or 128 x 128 tile (block_rows 128).  colwise: also the cast of each matrix
    transposed, from the same pass over x.  N % 16 == 0; colwise also
    M % 16 == 0."""
    shape = x.shape
    if len(shape) not in (2, 3):
        raise ValueError("x must be [M, N] or [B, M, N]")
    if not x.is_cuda or not x.is_contiguous():
        raise ValueError("tensors passed to libnvfp4 must be contiguous CUDA tensors")
    dtype = _DTYPES.get(x.dtype)
    if dtype is None:
        raise TypeError(f"quantize_fp8 takes bfloat16 or float32 input, got {x.dtype}")
    lead, (M, N) = tuple(shape[:-2]), shape[-2:]
    dev = x.device
    row = col = None
    pointers = [None] * 4
    if rowwise:
        data = torch.empty(shape, dtype=CODES, device=dev)
        scale = torch.empty(_scale_shape(lead, M, N, block_rows), dtype=torch.float32, device=dev)
        row = FP8Operand(data, scale, block_rows)
        pointers[:2] = data.data_ptr(), scale.data_ptr()
    if colwise:
        data = torch.empty(lead + (N, M), dtype=CODES, device=dev)
        scale = torch.empty(_scale_shape(lead, N, M, block_rows), dtype=torch.float32, device=dev)
        col = FP8Operand(data, scale, block_rows)
        pointers[2:] = data.data_ptr(), scale.data_ptr()
    call("nvfp4_fp8_quantize", dev, x.data_ptr(), dtype, lead[0] if lead else 1, M, N, block_rows, *pointers,
         (ROWWISE if rowwise else 0) | (COLWISE if colwise else 0))
    return FP8Tensor(row, col)


def _check_operand(name: str, q: FP8Operand, dims: int) -> tuple:
    """(the codes' shape, their device); raises where codes and scales do not fit each other."""
    d, s, block_rows = q.data, q.scale, q.block_rows
    shape, dev = d.shape, d.device
    if d.dtype is not CODES or s.dtype is not torch.float32:
        raise TypeError(f"{name}: float8_e4m3fn codes and float32 scales, got {d.dtype} and {s.dtype}")
    if len(shape) != dims:
        raise ValueError(f"{name}: codes with {dims} dimensions, got {tuple(shape)}")
    rows, cols = shape[-2:]
    if block_rows == 1:
        want = ((cols + 127) // BLOCK, rows)
    elif block_rows == BLOCK:
        want = ((rows + 127) // BLOCK, (cols + 127) // BLOCK)
    else:
        raise ValueError(f"{name}: block_rows 1 or {BLOCK}, got {block_rows}")
    if s.shape != (want if dims == 2 else (shape[0], *want)):
        raise ValueError(f"{name}: scales {tuple(s.shape)} do not fit codes {tuple(shape)} with block_rows "
                         f"{block_rows}")
    if not (d.is_cuda and d.is_contiguous() and s.is_contiguous()):
        raise ValueError("tensors passed to libnvfp4 must be contiguous CUDA tensors")
    if s.device != dev:
        raise ValueError(f"{name}: codes and scales on one device")
    return shape, dev


def _output(out: torch.Tensor | None, shape: tuple, dtype: torch.dtype, dev: torch.device) -> tuple:
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=dev)
    elif out.shape != shape or out.device != dev or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous {shape} tensor on {dev}")
    code = _DTYPES.get(out.dtype)
    if code is None:
        raise TypeError(f"products are bfloat16 or float32, not {out.dtype}")
    return out, code


def _check_pair(a: FP8Operand, b: FP8Operand, b_dims: int) -> tuple:
    a_shape, dev = _check_operand("a", a, 2)
    b_shape, b_dev = _check_operand("b", b, b_dims)
    if a.block_rows != 1:
        raise ValueError("a needs block_rows 1")
    if a_shape[-1] != b_shape[-1]:
        raise ValueError(f"the last dimensions of a {tuple(a_shape)} and b {tuple(b_shape)} differ")
    if dev != b_dev:
        raise ValueError("a and b on one device")
    return a_shape, b_shape, dev


def _check_offsets(offsets: torch.Tensor, dev: torch.device) -> None:
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or offsets.numel() < 2:
        raise TypeError("offsets: an int32 vector of experts + 1 entries")
    if offsets.device != dev or not offsets.is_contiguous():
        raise ValueError("offsets must be contiguous, on the operands' device")


def matmul_fp8(a: FP8Operand, b: FP8Operand, out_dtype: torch.dtype = torch.bfloat16,
               out: torch.Tensor | None = None) -> torch.Tensor:
    """a [M, K] times b [N, K] transposed: [M, N] in bfloat16 or float32.

    a has block_rows 1, b 1 or 128.  Each block of 128 is summed on the tensor
    cores in FP32, scaled, and added in FP32.  K % 16 == 0."""
    (M, K), (N, _), dev = _check_pair(a, b, 2)
    out, code = _output(out, (M, N), out_dtype, dev)
    call("nvfp4_fp8_matmul", dev, a.data.data_ptr(), a.scale.data_ptr(), b.data.data_ptr(), b.scale.data_ptr(),
         b.block_rows, M, N, K, out.data_ptr(), code)
    return out


def matmul_fp8_grouped(a: FP8Operand, b: FP8Operand, offsets: torch.Tensor,
                       out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """The product by expert: rows offsets[e] .. offsets[e+1] of a [R, K] times
    b[e] transposed, b [E, N, K]; [R, N], zero past offsets[E].  offsets: device
    int32, as ``TokenPlan.offsets`` (any alignment of the members); offsets that
    do not ascend from 0 to at most R give the value 4 from ``device_status``."""
    (R, K), (E, N, _), dev = _check_pair(a, b, 3)
    _check_offsets(offsets, dev)
    if offsets.numel() != E + 1:
        raise ValueError(f"{E} experts need {E + 1} offsets, got {offsets.numel()}")
    out, code = _output(out, (R, N), out_dtype, dev)
    call("nvfp4_fp8_matmul_grouped", dev, a.data.data_ptr(), a.scale.data_ptr(), b.data.data_ptr(), b.scale.data_ptr(),
         b.block_rows, R, N, K, E, offsets.data_ptr(), out.data_ptr(), code)
    return out


def matmul_fp8_grouped_wgrad(a: FP8Operand, b: FP8Operand, offsets: torch.Tensor,
                             out_dtype: torch.dtype = torch.float32, out: torch.Tensor | None = None) -> torch.Tensor:
    """The experts' weight gradients: out[e] = a[:, member e] times b[:, member
    e] transposed, a [N, R] and b [K, R] the column-wise casts of the output
    gradient and the input; [E, N, K], zero for an empty member.  Every offset
    a multiple of 128 (``dispatch_tokens`` with align=128), or the last one R:
    others give a wrong result and the value 4 from ``device_status``."""
    (N, R), (K, _), dev = _check_pair(a, b, 2)
    if b.block_rows != 1:
        raise ValueError("b needs block_rows 1")
    _check_offsets(offsets, dev)
    E = offsets.numel() - 1
    out, code = _output(out, (E, N, K), out_dtype, dev)
    call("nvfp4_fp8_matmul_grouped_wgrad", dev, a.data.data_ptr(), a.scale.data_ptr(), b.data.data_ptr(),
         b.scale.data_ptr(), N, K, R, E, offsets.data_ptr(), out.data_ptr(), code)
    return out
