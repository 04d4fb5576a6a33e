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

from . import BF16, FP32, _OnDevice, _lib

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


def _stream(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _dtype(t: torch.Tensor, name: str) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return FP32
    raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")


def _check(t: torch.Tensor, name: str, dims: int, device: torch.device) -> None:
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {tuple(t.shape)}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("tensors passed to libnvfp4 must be contiguous CUDA tensors")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, like the other tensors of the call")


def _empty_plan(ids: torch.Tensor, num_experts: int, align: int) -> tuple[TokenPlan, torch.Tensor | None]:
    dev = ids.device
    if ids.dtype != torch.int32:
        raise TypeError(f"expert_ids must be int32, got {ids.dtype}")
    if num_experts < 1 or num_experts > _lib.MAX_EXPERTS or align < 1:
        raise ValueError(f"1 to {_lib.MAX_EXPERTS} experts and align >= 1")
    slots = ids.numel()
    rows = (slots + num_experts * (align - 1)) // align * align
    # one allocation for the three maps, each starting on 16 bytes
    n0 = (num_experts + 1 + 3) // 4 * 4
    n1 = (slots + 3) // 4 * 4
    maps = torch.empty(n0 + n1 + rows, dtype=torch.int32, device=dev)
    plan = TokenPlan(maps[:num_experts + 1], maps[n0:n0 + slots].view(ids.shape), maps[n0 + n1:])
    scratch = None
    if slots > SORT_CHUNK:
        scratch = torch.empty(-(-slots // SORT_CHUNK) * num_experts, dtype=torch.int32, device=dev)
    return plan, scratch


def sort_tokens(expert_ids: torch.Tensor, num_experts: int, align: int = 1) -> TokenPlan:
    """Places the choices expert_ids [T, topk] (int32) in stable order of their
    expert, every expert's member padded to a multiple of ``align`` rows."""
    _check(expert_ids, "expert_ids", 2, expert_ids.device)
    plan, scratch = _empty_plan(expert_ids, num_experts, align)
    T, topk = expert_ids.shape
    with _OnDevice(expert_ids.device):
        rc = _lib.load().nvfp4_sort_tokens(
            expert_ids.data_ptr(), T, topk, num_experts, align, plan.offsets.data_ptr(), plan.row_of_slot.data_ptr(),
            plan.slot_of_row.data_ptr(), plan.rows, None if scratch is None else scratch.data_ptr(),
            0 if scratch is None else 4 * scratch.numel(), _stream(expert_ids.device))
    _lib.check(rc, "nvfp4_sort_tokens")
    return plan


def _check_plan(plan: TokenPlan, device: torch.device) -> None:
    _check(plan.row_of_slot, "plan.row_of_slot", 2, device)
    _check(plan.slot_of_row, "plan.slot_of_row", 1, device)
    if plan.row_of_slot.dtype != torch.int32 or plan.slot_of_row.dtype != torch.int32:
        raise TypeError("the maps of a plan are int32")


def gather_tokens(x: torch.Tensor, plan: TokenPlan) -> torch.Tensor:
    """x [T, H] -> [rows, H]: the token of each row, zero for padding."""
    _check(x, "x", 2, x.device)
    _check_plan(plan, x.device)
    T, H = x.shape
    if plan.row_of_slot.shape[0] != T:
        raise ValueError(f"the plan is for {plan.row_of_slot.shape[0]} tokens, x has {T}")
    out = torch.empty((plan.rows, H), dtype=x.dtype, device=x.device)
    with _OnDevice(x.device):
        rc = _lib.load().nvfp4_gather_tokens(x.data_ptr(), _dtype(x, "x"), T, H, plan.topk,
                                             plan.row_of_slot.data_ptr(), plan.slot_of_row.data_ptr(), plan.rows,
                                             out.data_ptr(), _stream(x.device))
    _lib.check(rc, "nvfp4_gather_tokens")
    return out


def dispatch_tokens(x: torch.Tensor, expert_ids: torch.Tensor, num_experts: int,
                    align: int = 1) -> tuple[torch.Tensor, TokenPlan]:
    """``sort_tokens`` and ``gather_tokens`` in one call: (rows, plan)."""
    _check(x, "x", 2, x.device)
    _check(expert_ids, "expert_ids", 2, x.device)
    T, H = x.shape
    if expert_ids.shape[0] != T:
        raise ValueError(f"expert_ids for {expert_ids.shape[0]} tokens, x has {T}")
    code = _dtype(x, "x")
    plan, scratch = _empty_plan(expert_ids, num_experts, align)
    rows = plan.slot_of_row.shape[0]
    out = torch.empty((rows, H), dtype=x.dtype, device=x.device)
    with _OnDevice(x.device):
        rc = _lib.load().nvfp4_dispatch_tokens(
            x.data_ptr(), code, T, H, expert_ids.data_ptr(), expert_ids.shape[1], num_experts, align,
            plan.offsets.data_ptr(), plan.row_of_slot.data_ptr(), plan.slot_of_row.data_ptr(), rows, out.data_ptr(),
            None if scratch is None else scratch.data_ptr(), 0 if scratch is None else 4 * scratch.numel(),
            _stream(x.device))
    _lib.check(rc, "nvfp4_dispatch_tokens")
    return out, plan


def _check_weights(weights: torch.Tensor | None, plan: TokenPlan, device: torch.device) -> None:
    if weights is None:
        return
    _check(weights, "weights", 2, device)
    if weights.dtype != torch.float32 or weights.shape != plan.row_of_slot.shape:
        raise ValueError(f"weights must be float32 {tuple(plan.row_of_slot.shape)}")


def combine_tokens(rows: torch.Tensor, plan: TokenPlan, weights: torch.Tensor | None = None) -> torch.Tensor:
    """rows [R, H] -> [T, H]: y[t] = sum_j weights[t, j] rows[row of (t, j)],
    summed in FP32 and rounded once; a dropped choice adds nothing.  weights:
    float32 [T, topk], or None for 1."""
    _check(rows, "rows", 2, rows.device)
    _check_plan(plan, rows.device)
    _check_weights(weights, plan, rows.device)
    R, H = rows.shape
    if R != plan.slot_of_row.shape[0]:
        raise ValueError(f"the plan has {plan.rows} rows, got {R}")
    T, topk = plan.row_of_slot.shape
    y = torch.empty((T, H), dtype=rows.dtype, device=rows.device)
    with _OnDevice(rows.device):
        rc = _lib.load().nvfp4_combine_tokens(rows.data_ptr(), _dtype(rows, "rows"), T, H, topk,
                                              plan.row_of_slot.data_ptr(), R,
                                              None if weights is None else weights.data_ptr(), y.data_ptr(),
                                              _stream(rows.device))
    _lib.check(rc, "nvfp4_combine_tokens")
    return y


def gather_tokens_grad(drows: torch.Tensor, plan: TokenPlan) -> torch.Tensor:
    """Gradient of ``gather_tokens``: the sum of each token's rows."""
    return combine_tokens(drows, plan, None)


def combine_tokens_grad(dy: torch.Tensor, rows: torch.Tensor, plan: TokenPlan,
                        weights: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """Gradient of ``combine_tokens``: (drows [R, H], dweights [T, topk]).
    drows is zero for padding rows, dweights for dropped choices."""
    _check(dy, "dy", 2, dy.device)
    _check(rows, "rows", 2, dy.device)
    _check_plan(plan, dy.device)
    _check_weights(weights, plan, dy.device)
    T, topk = plan.row_of_slot.shape
    R, H = rows.shape
    if R != plan.slot_of_row.shape[0] or dy.shape != (T, H):
        raise ValueError(f"dy must be [{T}, {H}] and rows [{plan.rows}, {H}], got {tuple(dy.shape)}, {tuple(rows.shape)}")
    if dy.dtype != rows.dtype:
        raise TypeError(f"dy and rows of one type, got {dy.dtype} and {rows.dtype}")
    drows = torch.empty_like(rows)
    dweights = torch.empty((T, topk), dtype=torch.float32, device=dy.device)
    with _OnDevice(dy.device):
        rc = _lib.load().nvfp4_combine_tokens_grad(
            dy.data_ptr(), rows.data_ptr(), _dtype(dy, "dy"), T, H, topk, plan.row_of_slot.data_ptr(),
            plan.slot_of_row.data_ptr(), R, None if weights is None else weights.data_ptr(), drows.data_ptr(),
            dweights.data_ptr(), _stream(dy.device))
    _lib.check(rc, "nvfp4_combine_tokens_grad")
    return drows, dweights
