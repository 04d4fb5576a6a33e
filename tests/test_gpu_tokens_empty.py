"""A batch of no tokens: the rows that padding leaves are zero, and nothing outside the outputs is written."""
import pytest
import torch

import nvfp4_block_scaled_amax_gb300 as nv
from nvfp4_block_scaled_amax_gb300 import BF16, FP32
from nvfp4_block_scaled_amax_gb300._call import call
from nvfp4_block_scaled_amax_gb300.experts import expert_layer, expert_layer_grad

pytestmark = pytest.mark.gpu

CODE = {torch.bfloat16: BF16, torch.float32: FP32}
GUARD = 64  # rows of a foreign value on both sides of an output: more than a warp or CTA looks at in one go
FOREIGN = 7.0


def guarded(rows, H, dtype):
    """(storage, the rows in the middle of it)"""
    storage = torch.full((rows + 2 * GUARD, H), FOREIGN, dtype=dtype, device="cuda")
    return storage, storage[GUARD:GUARD + rows]


def check_zero_inside_only(storage, rows):
    assert bool((storage[:GUARD] == FOREIGN).all()) and bool((storage[GUARD + rows:] == FOREIGN).all())
    assert bool((storage[GUARD:GUARD + rows] == 0).all())


# rows 48 and 384, and on both sides of the 6144 rows up to which sort and gather are one launch; members' ends that
# are multiples of 8 and 32 and ends that are not
SIZES = [(4, 16), (4, 128), (3, 100), (48, 128), (49, 128), (64, 128), (7, 1013)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E,align", SIZES)
def test_gather_and_dispatch_of_no_tokens(E, align, dtype):
    H, topk = 72, 2
    x = torch.empty(0, H, dtype=dtype, device="cuda")
    ids = torch.empty(0, topk, dtype=torch.int32, device="cuda")
    plan = nv.sort_tokens(ids, E, align=align)
    rows = E * (align - 1) // align * align
    assert plan.rows == rows and plan.offsets.tolist() == [0] * (E + 1) and bool((plan.slot_of_row == -1).all())

    storage, out = guarded(rows, H, dtype)
    call("nvfp4_gather_tokens", x.device, x.data_ptr(), CODE[dtype], 0, H, topk, plan.row_of_slot.data_ptr(),
         plan.slot_of_row.data_ptr(), rows, out.data_ptr())
    check_zero_inside_only(storage, rows)

    storage, out = guarded(rows, H, dtype)
    offsets, slot_of_row = torch.full_like(plan.offsets, 9), torch.full_like(plan.slot_of_row, 9)
    call("nvfp4_dispatch_tokens", x.device, x.data_ptr(), CODE[dtype], 0, H, ids.data_ptr(), topk, E, align,
         offsets.data_ptr(), plan.row_of_slot.data_ptr(), slot_of_row.data_ptr(), rows, out.data_ptr(), None, 0)
    check_zero_inside_only(storage, rows)
    assert torch.equal(offsets, plan.offsets) and torch.equal(slot_of_row, plan.slot_of_row)

    assert nv.gather_tokens(x, plan).shape == (rows, H) and nv.dispatch_tokens(x, ids, E, align=align)[0].shape == (rows, H)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E,align", SIZES)
def test_combine_and_its_gradient_of_no_tokens(E, align, dtype):
    H, topk = 72, 3
    dy = torch.empty(0, H, dtype=dtype, device="cuda")
    plan = nv.sort_tokens(torch.empty(0, topk, dtype=torch.int32, device="cuda"), E, align=align)
    rows_in = torch.full((plan.rows, H), float("nan"), dtype=dtype, device="cuda")  # never read
    weights = torch.empty(0, topk, device="cuda")
    assert nv.combine_tokens(rows_in, plan, weights).shape == (0, H)
    assert nv.gather_tokens_grad(rows_in, plan).shape == (0, H)

    for w in (None, weights):
        storage, drows = guarded(plan.rows, H, dtype)
        dweights = torch.full((8,), FOREIGN, device="cuda")
        call("nvfp4_combine_tokens_grad", dy.device, dy.data_ptr(), rows_in.data_ptr(), CODE[dtype], 0, H, topk,
             plan.row_of_slot.data_ptr(), plan.slot_of_row.data_ptr(), plan.rows, None if w is None else w.data_ptr(),
             drows.data_ptr(), dweights.data_ptr())
        check_zero_inside_only(storage, plan.rows)
        assert bool((dweights == FOREIGN).all())
    drows, dw = nv.combine_tokens_grad(dy, rows_in, plan, weights)
    assert bool((drows == 0).all()) and dw.shape == (0, topk)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E", [1, 3, 64])
def test_expert_layer_of_no_tokens(E, dtype):
    """As on a rank that a batch sends no token to: no output rows, zero weight gradients, nothing else changed."""
    N, K, topk = 144, 272, 2
    x, dy = (torch.empty(0, n, dtype=dtype, device="cuda") for n in (K, N))
    ids, gates = torch.empty(0, topk, dtype=torch.int32, device="cuda"), torch.empty(0, topk, device="cuda")
    w = torch.randn(E, N, K, device="cuda", dtype=dtype)
    kept = w.clone()
    y, saved = expert_layer(x, w, ids, gates)
    dx, dw, dg = expert_layer_grad(dy, saved)
    assert y.shape == (0, N) and dx.shape == (0, K) and dg.shape == (0, topk)
    assert dw.shape == (E, N, K) and bool((dw == 0).all())
    assert expert_layer(x, w, ids, gates, training=False)[0].shape == (0, N)
    assert torch.equal(w, kept) and nv.device_status() == 0
