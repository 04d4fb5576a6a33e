"""A layer of experts in 8 bits: a router's choices, one weight matrix per expert, and the sum over each token's choices.

    y, saved = expert_layer(x, weights, expert_ids, gates)
    dx, dweights, dgates = expert_layer_grad(dy, saved)

computes y[t] = sum_j gates[t, j] * weights[expert_ids[t, j]] @ x[t] and its gradients: the tokens are sorted by expert
(``dispatch_tokens``), cast to E4M3 rows and columns in one pass (``quantize_fp8``), multiplied by expert
(``matmul_fp8_grouped``) and joined (``combine_tokens``); backwards, the rows' gradient is cast the same way and gives the
input gradient (the column-wise weights) and the weight gradient (the column-wise activations).  Nothing waits for the
host: every size depends on the shapes alone.  As everywhere in this package autograd records nothing: the gradient is the
function beside the call.

For decoding, a whole layer of gated experts over 4-bit weights:

    up, down = quantize_experts(gate_up), quantize_experts(down)      # [E, 2 F, H], [E, H, F], once
    y = expert_mlp(x, up, down, expert_ids, gates)                    # two to five launches
"""
from __future__ import annotations

import ctypes
import functools
from dataclasses import dataclass

import torch

from . import FP4Operand, _lib, quantize_grouped, quantize_mxfp4
from ._call import call
from .fp4 import _check_operand, _struct
from .fp8 import BLOCK, FP8Tensor, matmul_fp8_grouped, matmul_fp8_grouped_wgrad, quantize_fp8
from .tokens import TokenPlan, combine_tokens, combine_tokens_grad, dispatch_tokens, gather_tokens_grad


@dataclass
class ExpertSaved:
    """What the gradient needs of the forward pass."""
    plan: TokenPlan
    gates: torch.Tensor
    rows: FP8Tensor      # the sorted tokens
    weights: FP8Tensor
    rows_out: torch.Tensor


def expert_layer(x: torch.Tensor, weights: torch.Tensor | FP8Tensor, expert_ids: torch.Tensor, gates: torch.Tensor,
                 training: bool = True) -> tuple[torch.Tensor, ExpertSaved | None]:
    """x [T, K] bfloat16, weights [E, N, K] (bfloat16 or float32, or their cast with block_rows 128), expert_ids int32
    and gates float32 [T, topk].  training: also cast the columns the gradients need, with members padded to 128 rows
    (K, N multiples of 16); otherwise the members are not padded and nothing is saved."""
    if isinstance(weights, torch.Tensor):
        weights = quantize_fp8(weights, block_rows=BLOCK, colwise=training)
    elif training and weights.col is None:
        raise ValueError("the gradients need the column-wise cast of the weights: quantize_fp8(..., colwise=True)")
    E = weights.row.data.shape[0]
    rows, plan = dispatch_tokens(x, expert_ids, E, align=BLOCK if training else 1)
    q = quantize_fp8(rows, colwise=training)
    rows_out = matmul_fp8_grouped(q.row, weights.row, plan.offsets, out_dtype=x.dtype)
    y = combine_tokens(rows_out, plan, gates)
    return y, ExpertSaved(plan, gates, q, weights, rows_out) if training else None


def expert_layer_grad(dy: torch.Tensor, saved: ExpertSaved) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(dx [T, K] in dy's type, dweights [E, N, K] float32, dgates [T, topk] float32)."""
    plan = saved.plan
    drows_out, dgates = combine_tokens_grad(dy, saved.rows_out, plan, saved.gates)
    q = quantize_fp8(drows_out, colwise=True)
    drows = matmul_fp8_grouped(q.row, saved.weights.col, plan.offsets, out_dtype=dy.dtype)
    dweights = matmul_fp8_grouped_wgrad(q.col, saved.rows.col, plan.offsets)
    return gather_tokens_grad(drows, plan), dweights, dgates


def quantize_experts(weights: torch.Tensor, block: int = 16) -> FP4Operand:
    """Casts a stack of weight matrices [E, N, K] (bfloat16 or float32) to 4 bits along K for ``expert_mlp``: NVFP4 with
    an amax for each matrix (block 16, N % 8 == 0) or MXFP4 (block 32).  K % 32 == 0.  For weights, ahead of use: it
    makes several calls."""
    if weights.dim() != 3:
        raise ValueError("weights must be [E, N, K]")
    E, N, K = weights.shape
    if K % 32:
        raise ValueError("the contracted dimension must be a multiple of 32")
    if not weights.is_contiguous():
        raise ValueError("tensors passed to libnvfp4 must be contiguous CUDA tensors")
    if block == 32:
        q = quantize_mxfp4(weights.view(E * N, K)).row
        return FP4Operand(q.data.view(E, N, K // 2), q.scale.view(E, N, K // 32), None, 32)
    if block != 16:
        raise ValueError(f"block 16 (NVFP4) or 32 (MXFP4), got {block}")
    if N % 8:
        raise ValueError("NVFP4 experts need a multiple of 8 rows")
    dev = weights.device
    data = torch.empty((E, N, K // 2), dtype=torch.uint8, device=dev)
    scale = torch.empty((E, N, K // 16), dtype=torch.uint8, device=dev)
    amax = torch.zeros((E, 4), dtype=torch.float32, device=dev)  # (each at a 16-byte boundary, as the cast writes them)
    from . import NVFP4Tensor
    for e0 in range(0, E if N * K else 0, _lib.MAX_GROUPS):
        members = range(e0, min(E, e0 + _lib.MAX_GROUPS))
        outs = [NVFP4Tensor(N, K, data[e], scale[e].view(-1), amax[e, :1]) for e in members]
        quantize_grouped(weights[e0:members.stop].view(-1, K), [N] * len(members), "1d", colwise=False, out=outs)
    return FP4Operand(data, scale, amax[:, 0].contiguous(), 16)


@functools.lru_cache(maxsize=256)
def _mlp_workspace(T: int, topk: int, E: int, H: int, F: int, block: int) -> int:
    n = ctypes.c_size_t(0)
    _lib.check(_lib.load().nvfp4_expert_mlp_workspace(T, topk, E, H, F, block, ctypes.byref(n)),
               "nvfp4_expert_mlp_workspace")
    return n.value


def expert_mlp(x: torch.Tensor, up: FP4Operand, down: FP4Operand, expert_ids: torch.Tensor, gates: torch.Tensor,
               out: torch.Tensor | None = None) -> torch.Tensor:
    """y[t] = sum_j gates[t, j] * down[e] @ (silu(gate[e] @ x[t]) * (up[e] @ x[t])), e = expert_ids[t, j], for a few
    tokens: x [T, H] bfloat16, expert_ids int32 and gates float32 [T, topk], up [E, 2 F, H] (an expert's gate rows, then
    its up rows) and down [E, H, F] 4-bit operands of one format with compact scales (``quantize_experts``).  Ids outside
    0 .. E - 1 are dropped.  T * topk <= 1024; H and F multiples of 32, at most 10240.  Sums are float32; what x and the
    hidden values are held in leaves at most 2^-22 of the largest value of each of their blocks (NVFP4: or 2^-39 of their
    row's), whatever the weights' amaxes.  An expert's weights are read again for every 14 of its tokens (8 where experts have few), so that many tokens
    an expert are not what this is for; ``expert_layer`` has no such limit, over weights in 8 bits."""
    E, F2, H = _check_operand("up", up, 3)
    Ed, Hd, F = _check_operand("down", down, 3)
    x_shape, ids_shape, dev = x.shape, expert_ids.shape, x.device
    if x.dtype is not torch.bfloat16 or gates.dtype is not torch.float32 or expert_ids.dtype is not torch.int32:
        raise TypeError(f"bfloat16 x, float32 gates and int32 expert_ids, got {x.dtype}, {gates.dtype} and "
                        f"{expert_ids.dtype}")
    if len(x_shape) != 2 or len(ids_shape) != 2 or gates.shape != ids_shape or ids_shape[0] != x_shape[0]:
        raise ValueError("x [T, H], expert_ids and gates [T, topk]")
    T, topk = ids_shape
    if Ed != E or Hd != H or F2 != 2 * F or x_shape[1] != H or up.block != down.block:
        raise ValueError(f"up [E, 2 F, H] and down [E, H, F] of one format for x [T, H], got {(E, F2, H)} (block "
                         f"{up.block}), {(Ed, Hd, F)} (block {down.block}) and {tuple(x_shape)}")
    if up.swizzled or down.swizzled:
        raise ValueError("expert_mlp takes compact scales")
    if T * topk > _lib.MAX_MLP_SLOTS or not 1 <= topk <= _lib.MAX_TOPK:
        raise ValueError(f"expert_mlp takes up to {_lib.MAX_MLP_SLOTS} choices, up to {_lib.MAX_TOPK} a token, got {T} x "
                         f"{topk}")
    if max(H, F) > _lib.MAX_MLP_WIDTH or not 1 <= E <= _lib.MAX_EXPERTS:
        raise ValueError(f"expert_mlp takes sizes up to {_lib.MAX_MLP_WIDTH} and up to {_lib.MAX_EXPERTS} experts")
    index = x.get_device()
    if index < 0 or not (x.is_contiguous() and expert_ids.is_contiguous() and gates.is_contiguous()) or \
            expert_ids.get_device() != index or gates.get_device() != index:
        raise ValueError("tensors passed to libnvfp4 must be contiguous CUDA tensors, on one device")
    if up.data.get_device() != index or down.data.get_device() != index:
        raise ValueError("weights and x on one device")
    if out is None:
        out = torch.empty_like(x)
    elif out.shape != x_shape or out.dtype != x.dtype or out.device != dev or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous bfloat16 {tuple(x_shape)} tensor on {dev}")
    need = _mlp_workspace(T, topk, E, H, F, up.block)
    work = torch.empty(need, dtype=torch.uint8, device=dev)
    call("nvfp4_expert_mlp", dev, x.data_ptr(), T, H, F, _struct(up, E), _struct(down, E), up.block,
         expert_ids.data_ptr(), gates.data_ptr(), topk, E, work.data_ptr(), need, out.data_ptr())
    return out
