"""The gated expert layer on activations that are small beside others of their block."""
import pytest
import torch

import nvfp4_block_scaled_amax_gb300 as nv

pytestmark = pytest.mark.gpu

U32, U16 = 2.0 ** -24, 2.0 ** -8


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("T,topk,E", [(1, 1, 1), (2, 2, 4), (1, 9, 12), (5, 2, 4), (13, 4, 16), (40, 3, 4)])
def test_small_elements_of_a_block(T, topk, E, block):
    """Every output is one element of x times a constant: row f of the gate weights picks x[0], of the up weights x[f], of the
    down weights h[f].  The elements of a block reach from its largest down to 2^-14 of it.

    A block's scale s is at most 9 / 8 of a sixth of its largest element (the next E4M3 number) or a third of it (the next
    power of two), and eight terms leave s 2^-21, of x and then of h; an NVFP4 block below 2^-19 of its row's largest there
    is none.  The sums have one element that is not zero, in each of eight columns, so they and SiLU cost a handful of
    roundings in 32 bits; the result is rounded to BF16 once."""
    H = F = 160
    code = 2                                                       # 1.0
    up, down = torch.zeros(E, 2 * F, H, dtype=torch.uint8), torch.zeros(E, H, F, dtype=torch.uint8)
    f = torch.arange(F)
    up[:, :F, 0], up[:, F + f, f], down[:, f, f] = code, code, code
    def operand(codes):
        one = torch.full((*codes.shape[:2], codes.shape[2] // block), 0x38 if block == 16 else 127, dtype=torch.uint8)
        amax = torch.full((E,), 2688.0).cuda() if block == 16 else None
        return nv.FP4Operand((codes[..., ::2] | codes[..., 1::2] << 4).cuda(), one.cuda(), amax, block)
    g = torch.Generator().manual_seed(T)
    x = (torch.rand(T, H, generator=g) + 1) * 2.0 ** -torch.randint(0, 15, (T, H), generator=g)
    x = x * torch.where(torch.rand(T, H, generator=g) < 0.5, 1.0, -1.0)
    x[:, ::16] = 1.0 + torch.rand(T, H // 16, generator=g)         # the largest
    x = x.bfloat16()
    ids = torch.randint(0, E, (T, topk), generator=g, dtype=torch.int32)
    gates = torch.zeros(T, topk)
    gates[:, 0] = 1.0
    y = nv.expert_mlp(x.cuda(), operand(up), operand(down), ids.cuda(), gates.cuda()).cpu().double()
    v = x.double()
    left = 2.0 ** -21 * (1.125 / 6 if block == 16 else 1 / 3)
    largest = lambda t: t.abs().view(T, -1, block).amax(2).repeat_interleave(block, 1)  # noqa: E731
    act = v[:, :1] / (1 + torch.exp(-v[:, :1]))
    dx = left * largest(v)
    h = act * v
    dh = act * dx + 1.1 * dx[:, :1] * (v.abs() + dx) + 16 * U32 * h.abs()
    dh = dh + left * largest(h.abs() + dh)
    off = dh + 8 * U32 * h.abs()
    assert bool(((y - h).abs() <= off * 1.01 + U16 * (h.abs() + off)).all())
    assert nv.device_status() == 0
