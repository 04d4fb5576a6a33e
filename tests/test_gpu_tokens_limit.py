"""The sort at the largest sizes it takes: members that end just below row 2^31."""
import pytest
import torch

import nvfp4_block_scaled_amax_gb300 as nv

pytestmark = [pytest.mark.gpu, pytest.mark.slow]


@pytest.mark.parametrize("T,align", [((1 << 31) - 1, 1),               # no padding, the last row is 2^31 - 2
                                     (((1 << 31) - 1) // 600 * 600 - 5, 600)])  # five rows of padding, members by the CTA
def test_sort_of_a_member_that_ends_below_two_to_the_31(T, align):
    ids = torch.zeros(T, 1, device="cuda", dtype=torch.int32)
    plan = nv.sort_tokens(ids, 1, align=align)
    rows = -(-T // align) * align
    assert plan.offsets.tolist() == [0, rows] and plan.rows == rows
    for s in range(0, T, 1 << 28):
        e = min(s + (1 << 28), T)
        want = torch.arange(s, e, device="cuda", dtype=torch.int32)
        assert torch.equal(plan.row_of_slot[s:e, 0], want) and torch.equal(plan.slot_of_row[s:e], want)
    assert bool((plan.slot_of_row[T:] == -1).all())
    assert not bool(ids.any())
