"""Sizes that the sort does not take are refused with a message, before anything is allocated."""
import ctypes

import pytest
import torch

from nvfp4_block_scaled_amax_gb300 import _lib, tokens


def ids(T, topk):
    return torch.empty(T, topk, dtype=torch.int32, device="meta")  # a shape without memory


@pytest.mark.parametrize("T,topk,experts,align,what", [
    (4, 65, 8, 1, "64 choices"), (4, 0, 8, 1, "64 choices"), (4, 2, 0, 1, "experts"), (4, 2, 1025, 1, "experts"),
    (4, 2, 8, 0, "align"), (4, 2, 8, (1 << 20) + 1, "align"), (1 << 30, 2, 8, 1, "2\\^31"),
    ((1 << 31) - 8, 1, 64, 128, "2\\^31")])
def test_refused_with_a_message(T, topk, experts, align, what):
    with pytest.raises(ValueError, match=what):
        tokens._empty_plan(ids(T, topk), experts, align)
    # and by the C entry point
    rows, scratch = ctypes.c_int64(), ctypes.c_size_t()
    assert _lib.load().nvfp4_token_rows(T, topk, experts, align, ctypes.byref(rows), ctypes.byref(scratch)) == 2


@pytest.mark.parametrize("T,topk,experts,align", [(4, 64, 1024, 1 << 10), (4, 1, 1, 1 << 20), (0, 2, 4, 128)])
def test_taken_at_the_limits(T, topk, experts, align):
    plan, rows, pointer, size, _ = tokens._empty_plan(ids(T, topk), experts, align)
    want, scratch = ctypes.c_int64(), ctypes.c_size_t()
    assert _lib.load().nvfp4_token_rows(T, topk, experts, align, ctypes.byref(want), ctypes.byref(scratch)) == 0
    assert rows == want.value == plan.rows and size == scratch.value and pointer is None
