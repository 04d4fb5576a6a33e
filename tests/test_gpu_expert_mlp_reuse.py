"""The gated expert layer over inputs and a workspace that change from call to call, and at its limits."""
import pytest
import torch

import nvfp4_block_scaled_amax_gb300 as nv
from test_gpu_expert_mlp import check, stack

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("T,topk", [(1, 2), (2, 4), (12, 2), (40, 3)])
def test_inputs_written_just_before(T, topk, block):
    """The same memory for choices, gates and x, written by the kernels right before each call: every call sees its
    own, whatever earlier launches read ahead of time."""
    E, H, F, n = 9, 320, 160, 5
    up, _ = stack(E, 2 * F, H, block, 1, H ** -0.5)
    down, _ = stack(E, H, F, block, 2, F ** -0.5)
    g = torch.Generator().manual_seed(T)
    sets = [(torch.randn(T, H, generator=g).bfloat16().cuda(),
             torch.randint(-1, E if i else 1, (T, topk), generator=g, dtype=torch.int32).cuda(),
             torch.rand(T, topk, generator=g).cuda()) for i in range(n)]
    want = []
    for x, ids, gates in sets:
        want.append(nv.expert_mlp(x, up, down, ids, gates))
        torch.cuda.synchronize()
    x, ids, gates = (torch.empty_like(v) for v in sets[0])
    out = torch.empty(60, T, H, dtype=torch.bfloat16, device="cuda")
    order = torch.randint(0, n, (60,), generator=g).tolist()
    for k, i in enumerate(order):
        for to, v in zip((x, ids, gates), sets[i]):
            to.copy_(v)
        nv.expert_mlp(x, up, down, ids, gates, out=out[k])
    for k, i in enumerate(order):
        assert torch.equal(out[k], want[i])
    # the output in the place of the input
    x.copy_(sets[1][0])
    assert torch.equal(nv.expert_mlp(x, up, down, sets[1][1], sets[1][2], out=x), want[1])
    assert nv.device_status() == 0


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("T,topk,E,H,F", [(1024, 1, 3, 64, 32), (16, 64, 70, 64, 32), (512, 2, 1024, 32, 32),
                                          (1, 64, 1024, 96, 32)])
def test_limits(T, topk, E, H, F, block):
    """As many choices and experts as one call takes."""
    check(T, topk, E, H, F, block, seed=3)


def test_experts_without_elements():
    for block in (16, 32):
        for shape in ((2, 8, 0), (2, 0, 32)):
            q = nv.quantize_experts(torch.empty(shape, device="cuda"), block)
            assert q.data.shape == (shape[0], shape[1], shape[2] // 2) and q.scale.numel() == 0
            assert block == 32 or bool((q.amax == 0).all())
