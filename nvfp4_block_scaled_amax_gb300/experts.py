"""A layer of experts in 8 bits: a router's choices, one weight matrix per expert, and the sum over each token's choices.

    y, saved = expert_layer(x, weights, expert_ids, gates)
    dx, dweights, dgates = expert_layer_grad(dy, saved)

computes y[t] = sum_j gates[t, j] * weights[expert_ids[t, j]] @ x[t] and its gradients: the tokens are sorted by expert
(``dispatch_tokens``), cast to E4M3 rows and columns in one pass (``quantize_fp8``), multiplied by expert
(``matmul_fp8_grouped``) and joined (``combine_tokens``); backwards, the rows' gradient is cast the same way and gives the
input gradient (the column-wise weights) and the weight gradient (the column-wise activations).  Nothing waits for the
host: every size depends on the shapes alone.  As everywhere in this package autograd records nothing: the gradient is the
function beside the call.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

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
