"""The gated expert layer over NVFP4 and MXFP4 weights at its largest sizes, and with hidden values past FP32's range."""
import pytest
import torch

import nvfp4_block_scaled_amax_gb300 as nv
from test_gpu_fp4_large import random_operand

pytestmark = pytest.mark.gpu


def stack(E, n, k, seed, block):
    q = random_operand(E * n, k, seed, block)
    scale = q.scale if block == 16 else q.scale + 64             # bytes 0x30 .. 0x3F; as powers of two about 1
    return nv.FP4Operand(q.data.view(E, n, k // 2), scale.view(E, n, k // block),
                         torch.full((E,), 30.0, device="cuda") if block == 16 else None, block)


@pytest.mark.slow
@pytest.mark.parametrize("block", [16, 32])
def test_most_choices_of_the_widest_layer(block):
    """1024 choices, hidden and inner sizes of 10240: a token's result does not depend on where it stands among the others,
    and agrees with the same token alone, whose sums are shared otherwise (FP32's last bits, then one rounding to BF16)."""
    H = F = 10240
    up, down = stack(2, 2 * F, H, 1, block), stack(2, H, F, 2, block)
    x = (torch.randn(256, H, device="cuda") * (1.0 if block == 16 else 2.0 ** -8)).bfloat16()
    x = torch.cat([x, x.flip(0)])
    ids = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda").repeat(512, 1)
    gates = torch.tensor([[0.75, 0.25]], device="cuda").repeat(512, 1)
    y = nv.expert_mlp(x, up, down, ids, gates)
    assert bool(torch.isfinite(y).all()) and bool((y != 0).any(1).all())
    assert torch.equal(y[:256], y[256:].flip(0))
    for t in (0, 100, 255):
        one = nv.expert_mlp(x[t:t + 1], up, down, ids[:1], gates[:1]).double()
        assert float((y[t].double() - one[0]).norm() / one.norm()) < 2.0 ** -8
    assert nv.device_status() == 0


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("T", [2, 9, 30])
def test_hidden_values_past_the_range(T, block):
    """A token whose hidden values overflow gives NaN or infinities of its own and leaves the others as they are."""
    E, H, F = 3, 256, 96
    up, down = stack(E, 2 * F, H, 3, block), stack(E, H, F, 4, block)
    x = (torch.randn(T, H, device="cuda") * 2.0 ** -8).bfloat16()
    ids = torch.randint(0, E, (T, 2), device="cuda", dtype=torch.int32)
    gates = torch.rand(T, 2, device="cuda")
    want = nv.expert_mlp(x, up, down, ids, gates)
    assert bool(torch.isfinite(want).all())
    hot = x.clone()
    hot[T // 2] = hot[T // 2].float().sign().mul(1e30).bfloat16()
    y = nv.expert_mlp(hot, up, down, ids, gates)
    rest = [t for t in range(T) if t != T // 2]
    assert torch.equal(y[rest], want[rest]) and not bool(torch.isfinite(y[T // 2]).all())
    assert nv.device_status() == 0
