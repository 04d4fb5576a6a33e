"""A linear layer in 4 bits, forward and backward.

    y, saved = linear_layer(x, weight)              # x [T, K], weight [N, K]
    dx, dweight = linear_layer_grad(dy, saved)

computes y = x weight^T and its gradients on operands that are cast to 4 bits along what each product contracts: x and
the weight along K, and for the gradients (from the same pass over each) along T and N; dy along N and T.  Formats:
"mxfp4" (``quantize_mxfp4``) or "nvfp4" (``quantize``: 1x16 blocks of x and dy, 16x16 tiles of the weight, so that both
its casts agree).  As everywhere in this package autograd records nothing: the gradient is the function beside the call.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import NVFP4Tensor, quantize
from .fp4 import FP4Tensor, matmul_fp4, quantize_mxfp4


@dataclass
class LinearSaved:
    """What the gradient needs of the forward pass."""
    x: FP4Tensor | NVFP4Tensor
    weight: FP4Tensor | NVFP4Tensor
    format: str


def _cast(v: torch.Tensor, fmt: str, colwise: bool, mode: str) -> FP4Tensor | NVFP4Tensor:
    if v.dim() != 2:
        raise ValueError("a linear layer takes matrices")
    swizzled = v.shape[0] % 128 == 0 and v.shape[1] % 128 == 0 and v.numel() > 0
    if fmt == "mxfp4":
        return quantize_mxfp4(v, colwise=colwise, swizzled=swizzled)
    if fmt == "nvfp4":
        return quantize(v, mode, colwise=colwise, swizzled=swizzled)
    raise ValueError(f"unknown format {fmt!r}")


def quantize_linear(weight: torch.Tensor, format: str = "mxfp4", training: bool = True) -> FP4Tensor | NVFP4Tensor:
    """The casts of a weight [N, K] that ``linear_layer`` takes in its place."""
    return _cast(weight, format, training, "2d" if weight.dim() == 2 and weight.shape[0] % 16 == 0 else "1d")


def _weight_shape(weight: torch.Tensor | FP4Tensor | NVFP4Tensor) -> tuple[int, int]:
    if isinstance(weight, torch.Tensor):
        if weight.dim() != 2:
            raise ValueError("a linear layer takes matrices")
        return tuple(weight.shape)
    if weight.row is None:
        raise ValueError("the product needs the row-wise cast of the weight")
    N, half = weight.row.data.shape
    return N, 2 * half


def linear_layer(x: torch.Tensor, weight: torch.Tensor | FP4Tensor | NVFP4Tensor, format: str = "mxfp4",
                 training: bool = True) -> tuple[torch.Tensor, LinearSaved | None]:
    """y = x weight^T [T, N] in x's type, x [T, K] bfloat16 or float32, weight [N, K] or its casts
    (``quantize_linear``).  K a multiple of 32; training: T and N too, and what ``linear_layer_grad`` needs is kept."""
    N, K = _weight_shape(weight)
    if x.dim() != 2 or x.shape[1] != K:
        raise ValueError(f"x [T, {K}] for a weight [{N}, {K}], got {tuple(x.shape)}")
    if K % 32:
        raise ValueError(f"K must be a multiple of 32, got {K}")
    if training and (x.shape[0] % 32 or N % 32):
        raise ValueError(f"the gradients contract T and N: multiples of 32, got {x.shape[0]} and {N}")
    if isinstance(weight, torch.Tensor):
        weight = quantize_linear(weight, format, training)
    elif training and weight.col is None:
        raise ValueError("the gradients need the column-wise cast of the weight: quantize_linear(weight, training=True)")
    q = _cast(x, format, training, "1d")
    y = matmul_fp4(q.row, weight.row, out_dtype=x.dtype)
    return y, LinearSaved(q, weight, format) if training else None


def linear_layer_grad(dy: torch.Tensor, saved: LinearSaved) -> tuple[torch.Tensor, torch.Tensor]:
    """(dx [T, K] in dy's type, dweight [N, K] float32), dy [T, N]."""
    shape = saved.x.row.data.shape[0], saved.weight.row.data.shape[0]
    if dy.shape != shape:
        raise ValueError(f"dy must be {shape}, got {tuple(dy.shape)}")
    q = _cast(dy, saved.format, True, "1d")
    return matmul_fp4(q.row, saved.weight.col, out_dtype=dy.dtype), \
        matmul_fp4(q.col, saved.x.col, out_dtype=torch.float32)
