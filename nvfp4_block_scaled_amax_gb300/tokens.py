"""Tokens sorted by expert and joined again.

    rows, plan = dispatch_tokens(x, expert_ids, num_experts, align=128)
    ...                                            # per expert: plan.offsets[e] .. plan.offsets[e + 1]
    y = combine_tokens(rows_out, plan, weights)

``expert_ids`` [T, topk] are a router's choices; an id outside 0 .. num_experts
- 1 (-1, say) drops that choice.  Everything stays on the device: the number
of rows allocated depends on the shapes only, never on the ids.
"""
from __future__ import annotations

import torch

from . import BF16, FP32, _lib
from ._call import call

SORT_CHUNK = 2048  # slots up to which the sort needs no scratch


class TokenPlan:
    """Where each choice of the router went.

    offsets [experts + 1]: first row of each expert's member, and the end.
    row_of_slot [T, topk]: row of each choice, -1 if dropped.
    slot_of_row [rows]: choice (t * topk + j) of each row, -1 for padding.
    All int32, on the device.
    """
    __slots__ = ("offsets", "row_of_slot", "slot_of_row")

    def __init__(self, offsets: torch.Tensor, row_of_slot: torch.Tensor, slot_of_row: torch.Tensor):
        self.offsets, self.row_of_slot, self.slot_of_row = offsets, row_of_slot, slot_of_row

    @property
    def rows(self) -> int:
        return self.slot_of_row.shape[0]

    @property
    def topk(self) -> int:
        return self.row_of_slot.shape[1]


_DTYPES = {torch.bfloat16: BF16, torch.float32: FP32}


def _dtype(t: torch.Tensor, name: str) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    return code


def _check(t: torch.Tensor, name: str, dims: int, device: torch.device) -> tuple:
    shape = t.shape
    if len(shape) != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {tuple(shape)}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("tensors passed to libnvfp4 must be contiguous CUDA tensors")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, like the other tensors of the call")
    return shape


def _empty_plan(ids: torch.Tensor, num_experts: int, align: int) -> tuple:
    """(plan, rows, scratch pointer, scratch bytes, scratch): what a sort of ids writes."""
    dev, shape = ids.device, ids.shape
    if ids.dtype is not torch.int32:
        raise TypeError(f"expert_ids must be int32, got {ids.dtype}")
    if num_experts < 1 or num_experts > _lib.MAX_EXPERTS or align < 1 or align > _lib.MAX_ALIGN:
        raise ValueError(f"1 to {_lib.MAX_EXPERTS} experts and align 1 to {_lib.MAX_ALIGN}, got {num_experts} and {align}")
    if not 1 <= shape[1] <= _lib.MAX_TOPK:
        raise ValueError(f"expert_ids with 1 to {_lib.MAX_TOPK} choices a token, got {shape[1]}")
    slots = shape[0] * shape[1]
    rows = (slots + num_experts * (align - 1)) // align * align
    if slots >= 1 << 31 or rows >= 1 << 31:
        raise ValueError(f"choices and rows below 2^31, got {slots} and {rows}")
    plan = TokenPlan(torch.empty(num_experts + 1, dtype=torch.int32, device=dev),
                     torch.empty(shape, dtype=torch.int32, device=dev),
                     torch.empty(rows, dtype=torch.int32, device=dev))
    if slots <= SORT_CHUNK:
        return plan, rows, None, 0, None
    scratch = torch.empty(-(-slots // SORT_CHUNK) * num_experts, dtype=torch.int32, device=dev)
    return plan, rows, scratch.data_ptr(), 4 * scratch.numel(), scratch


def sort_tokens(expert_ids: torch.Tensor, num_experts: int, align: int = 1) -> TokenPlan:
    """Places the choices expert_ids [T, topk] (int32) in stable order of their
    expert, every expert's member padded to a multiple of ``align`` rows."""
    dev = expert_ids.device
    T, topk = _check(expert_ids, "expert_ids", 2, dev)
    plan, rows, scratch, size, _keep = _empty_plan(expert_ids, num_experts, align)
    call("nvfp4_sort_tokens", dev, expert_ids.data_ptr(), T, topk, num_experts, align, plan.offsets.data_ptr(),
         plan.row_of_slot.data_ptr(), plan.slot_of_row.data_ptr(), rows, scratch, size)
    return plan


def _check_plan(plan: TokenPlan, device: torch.device) -> tuple:
    """(tokens, topk, rows)"""
    at, slot = plan.row_of_slot, plan.slot_of_row
    T, topk = _check(at, "plan.row_of_slot", 2, device)
    rows, = _check(slot, "plan.slot_of_row", 1, device)
    if at.dtype is not torch.int32 or slot.dtype is not torch.int32:
        raise TypeError("the maps of a plan are int32")
    return T, topk, rows


def gather_tokens(x: torch.Tensor, plan: TokenPlan) -> torch.Tensor:
    """x [T, H] -> [rows, H]: the token of each row, zero for padding."""
    dev = x.device
    T, H = _check(x, "x", 2, dev)
    tokens, topk, rows = _check_plan(plan, dev)
    if tokens != T:
        raise ValueError(f"the plan is for {tokens} tokens, x has {T}")
    out = torch.empty((rows, H), dtype=x.dtype, device=dev)
    call("nvfp4_gather_tokens", dev, x.data_ptr(), _dtype(x, "x"), T, H, topk, plan.row_of_slot.data_ptr(),
         plan.slot_of_row.data_ptr(), rows, out.data_ptr())
    return out


def dispatch_tokens(x: torch.Tensor, expert_ids: torch.Tensor, num_experts: int,
                    align: int = 1) -> tuple[torch.Tensor, TokenPlan]:
    """``sort_tokens`` and ``gather_tokens`` in one call: (rows, plan)."""
    dev = x.device
    T, H = _check(x, "x", 2, dev)
    tokens, topk = _check(expert_ids, "expert_ids", 2, dev)
    if tokens != T:
        raise ValueError(f"expert_ids for {tokens} tokens, x has {T}")
    code = _dtype(x, "x")
    plan, rows, scratch, size, _keep = _empty_plan(expert_ids, num_experts, align)
    out = torch.empty((rows, H), dtype=x.dtype, device=dev)
    call("nvfp4_dispatch_tokens", dev, x.data_ptr(), code, T, H, expert_ids.data_ptr(), topk, num_experts, align,
         plan.offsets.data_ptr(), plan.row_of_slot.data_ptr(), plan.slot_of_row.data_ptr(), rows, out.data_ptr(),
         scratch, size)
    return out, plan


def _check_weights(weights: torch.Tensor | None, shape: tuple, device: torch.device) -> int | None:
    if weights is None:
        return None
    if _check(weights, "weights", 2, device) != shape or weights.dtype is not torch.float32:
        raise ValueError(f"weights must be float32 {shape}")
    return weights.data_ptr()


def combine_tokens(rows: torch.Tensor, plan: TokenPlan, weights: torch.Tensor | None = None) -> torch.Tensor:
    """rows [R, H] -> [T, H]: y[t] = sum_j weights[t, j] rows[row of (t, j)],
    summed in FP32 and rounded once; a dropped choice adds nothing.  weights:
    float32 [T, topk], or None for 1."""
    dev = rows.device
    R, H = _check(rows, "rows", 2, dev)
    T, topk, plan_rows = _check_plan(plan, dev)
    w = _check_weights(weights, (T, topk), dev)
    if R != plan_rows:
        raise ValueError(f"the plan has {plan_rows} rows, got {R}")
    y = torch.empty((T, H), dtype=rows.dtype, device=dev)
    call("nvfp4_combine_tokens", dev, rows.data_ptr(), _dtype(rows, "rows"), T, H, topk, plan.row_of_slot.data_ptr(), R,
         w, y.data_ptr())
    return y


def gather_tokens_grad(drows: torch.Tensor, plan: TokenPlan) -> torch.Tensor:
    """Gradient of ``gather_tokens``: the sum of each token's rows."""
    return combine_tokens(drows, plan, None)


def combine_tokens_grad(dy: torch.Tensor, rows: torch.Tensor, plan: TokenPlan,
                        weights: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """Gradient of ``combine_tokens``: (drows [R, H], dweights [T, topk]).
    drows is zero for padding rows, dweights for dropped choices."""
    dev = dy.device
    dy_shape = _check(dy, "dy", 2, dev)
    R, H = _check(rows, "rows", 2, dev)
    T, topk, plan_rows = _check_plan(plan, dev)
    w = _check_weights(weights, (T, topk), dev)
    if R != plan_rows or dy_shape != (T, H):
        raise ValueError(f"dy must be [{T}, {H}] and rows [{plan_rows}, {H}], got {tuple(dy_shape)}, {(R, H)}")
    if dy.dtype is not rows.dtype:
        raise TypeError(f"dy and rows of one type, got {dy.dtype} and {rows.dtype}")
    code = _dtype(dy, "dy")
    drows = torch.empty((R, H), dtype=rows.dtype, device=dev)
    dweights = torch.empty((T, topk), dtype=torch.float32, device=dev)
    call("nvfp4_combine_tokens_grad", dev, dy.data_ptr(), rows.data_ptr(), code, T, H, topk,
         plan.row_of_slot.data_ptr(), plan.slot_of_row.data_ptr(), R, w, drows.data_ptr(), dweights.data_ptr())
    return drows, dweights
