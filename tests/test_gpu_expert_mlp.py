"""The gated expert layer for a few tokens over 4-bit weights, against 64-bit arithmetic."""
import pytest
import torch

import nvfp4_block_scaled_amax_gb300 as nv
from fp4_testutil import random_parts, values

pytestmark = pytest.mark.gpu

U32, U16 = 2.0 ** -24, 2.0 ** -8


def stack(E, rows, cols, block, seed, std):
    """(operand, values [E, rows, cols]) of random matrices of about this deviation; NVFP4: an amax for each."""
    g = torch.Generator().manual_seed(seed)
    data = torch.randint(0, 256, (E, rows, cols // 2), generator=g, dtype=torch.uint8)
    if block == 32:
        scale = torch.randint(-3, 2, (E, rows, cols // 32), generator=g)
        scale = (scale + 127 + int(torch.tensor(std / 3).log2())).to(torch.uint8)
        amax = None
    else:
        scale = torch.randint(0x28, 0x50, (E, rows, cols // 16), generator=g, dtype=torch.uint8)
        amax = (torch.rand(E, generator=g) + 0.5) * 2688 * std / 6
    v = torch.stack([values(data[e], scale[e], None if amax is None else amax[e:e + 1], block) for e in range(E)])
    op = nv.FP4Operand(data.cuda(), scale.cuda(), None if amax is None else amax.cuda(), block)
    return op, v


def block_max(v, block):
    return v.abs().view(-1, block).amax(1).repeat_interleave(block)


def reference(x, up, down, ids, gates, block, amax):
    """(y, bound on the error) in 64 bits.

    x enters the products as six rows of E2M1 codes with one scale s for a block: the first is off by at most s, each
    later one by half its unit, s / 4 / 8^i, so s 2^-15 is left; s is at most the next E4M3 number above a sixth of the
    largest element (1/8 more, or the smallest one, 2^-9 of a unit that is at most 2^-10 of the row's largest), or the
    next power of two (a third of it).  A sum of n products in each of six columns is off by n U32 of the magnitudes,
    which the terms at most double.  The factor, SiLU (derivative below 1.1) and the product cost a handful of roundings;
    h is cut like x, its NVFP4 unit being taken from 2 (amax sum|x|)^2; then the same again."""
    T, H = x.shape
    F = down.shape[2]
    left = 2.0 ** -15 * (1.125 / 6 if block == 16 else 1 / 3)
    y, bound = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if not 0 <= e < up.shape[0]:
                continue
            v = x[t].double()
            dx = left * block_max(v, block) + (2.0 ** -34 * v.abs().max() if block == 16 else 0.0)
            s = up[e] @ v
            ds = up[e].abs() @ (dx + 2 * (H + 8) * U32 * v.abs())
            g, u, dg, du = s[:F], s[F:], ds[:F], ds[F:]
            act = g / (1 + torch.exp(-g))
            h = act * u
            dh = 1.1 * dg * (u.abs() + du) + act.abs() * du + 12 * U32 * h.abs()
            dh = dh + left * block_max(h.abs() + dh, block)
            if block == 16:
                dh = dh + 2.0 ** -34 * 2 * (float(amax[e]) * float(v.abs().sum())) ** 2
            w = float(gates[t, j])
            y[t] += w * (down[e] @ h)
            bound[t] += abs(w) * (down[e].abs() @ (dh + 2 * (F + 8) * U32 * h.abs()))
    return y, bound * 1.01 + U16 * (y.abs() + bound)


def check(T, topk, E, H, F, block, seed=0, ids=None):
    g = torch.Generator().manual_seed(seed)
    up, up_v = stack(E, 2 * F, H, block, seed + 1, H ** -0.5)
    down, down_v = stack(E, H, F, block, seed + 2, F ** -0.5)
    x = torch.randn(T, H, generator=g).bfloat16()
    if ids is None:
        ids = torch.randint(-1, E, (T, topk), generator=g, dtype=torch.int32)
    gates = torch.softmax(torch.randn(T, topk, generator=g), 1)
    args = (x.cuda(), up, down, ids.cuda(), gates.cuda())
    y = nv.expert_mlp(*args)
    want, bound = reference(x, up_v, down_v, ids, gates, block, None if up.amax is None else up.amax.cpu())
    assert bool(((y.cpu().double() - want).abs() <= bound).all())
    for _ in range(3):
        assert torch.equal(nv.expert_mlp(*args), y)  # whatever the order in which the CTAs finish
    assert nv.device_status() == 0
    return y


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("T,topk,E,H,F", [(1, 1, 1, 32, 32), (1, 2, 8, 256, 128), (3, 2, 4, 160, 96), (8, 2, 4, 512, 352),
                                          (9, 4, 6, 1184, 160), (16, 3, 5, 96, 1056), (17, 2, 3, 288, 256),
                                          (40, 2, 3, 256, 192), (64, 4, 32, 128, 64), (5, 8, 200, 64, 32),
                                          (1, 2, 4, 4096, 2048), (100, 1, 1, 64, 64),
                                          (13, 4, 16, 2720, 1184), (40, 2, 5, 1056, 5120), (2, 4, 6, 1184, 1056),
                                          (2, 1, 3, 10240, 64), (1, 8, 8, 320, 4096), (2, 2, 2, 64, 10240),
                                          (2, 4, 40, 2048, 512), (1, 9, 20, 256, 96)])
def test_layer(T, topk, E, H, F, block):
    check(T, topk, E, H, F, block, seed=T + H)


@pytest.mark.parametrize("block", [16, 32])
def test_ids(block):
    """Dropped choices, tokens without any, ids out of range, the same expert twice, one expert for all, none at all."""
    ids = torch.tensor([[-1, -1, -1], [2, 2, 2], [0, 5, 1], [7, -8, 3], [3, 1, 3]], dtype=torch.int32)
    y = check(5, 3, 4, 128, 96, block, ids=ids)
    assert bool((y[0] == 0).all())
    check(30, 2, 4, 128, 96, block, ids=torch.full((30, 2), 1, dtype=torch.int32))
    y = check(4, 2, 4, 128, 96, block, ids=torch.full((4, 2), -1, dtype=torch.int32))
    assert bool((y == 0).all())
    for rows in ([[-1, -1, -1]], [[3, 3, 3]], [[2, 9, -5]], [[-1, -1, 0], [-1, -1, -1]], [[1, 0, 1], [3, 1, 2]],
                 [[-1, -1, -1], [2, 2, 0]]):
        y = check(len(rows), 3, 4, 1536, 96, block, ids=torch.tensor(rows, dtype=torch.int32))
        for t, row in enumerate(rows):
            assert any(0 <= e < 4 for e in row) or bool((y[t] == 0).all())


@pytest.mark.parametrize("block", [16, 32])
def test_quantized_experts(block):
    """The casts' operands, as a user makes them; more experts than one grouped cast takes."""
    E, H, F, T = 70, 64, 32, 6
    g = torch.Generator().manual_seed(3)
    w1, w2 = torch.randn(E, 2 * F, H, generator=g) * 0.2, torch.randn(E, H, F, generator=g) * 0.2
    up, down = nv.quantize_experts(w1.bfloat16().cuda(), block), nv.quantize_experts(w2.cuda(), block)
    for op, w in ((up, w1.bfloat16()), (down, w2)):
        one = nv.quantize_experts(w[69:].contiguous().cuda(), block)
        assert torch.equal(op.data[69:], one.data) and torch.equal(op.scale[69:], one.scale)
        assert block == 32 or torch.equal(op.amax[69:], one.amax)
        assert block == 32 or torch.equal(op.amax.cpu(), w.float().abs().amax((1, 2)))
    vals = [torch.stack([values(o.data[e].cpu(), o.scale[e].cpu(), None if o.amax is None else o.amax[e:e + 1].cpu(), block)
                         for e in range(E)]) for o in (up, down)]
    x = torch.randn(T, H, generator=g).bfloat16()
    ids = torch.randint(0, E, (T, 2), generator=g, dtype=torch.int32)
    gates = torch.rand(T, 2, generator=g)
    y = nv.expert_mlp(x.cuda(), up, down, ids.cuda(), gates.cuda())
    want, bound = reference(x, *vals, ids, gates, block, None if up.amax is None else up.amax.cpu())
    assert bool(((y.cpu().double() - want).abs() <= bound).all())


@pytest.mark.parametrize("block", [16, 32])
def test_range_of_activations(block):
    """Large, tiny, infinite and NaN activations: each row its own scale, and no row touches another."""
    E, H, F = 2, 256, 64
    up, up_v = stack(E, 2 * F, H, block, 1, H ** -0.5)
    down, down_v = stack(E, H, F, block, 2, F ** -0.5)
    g = torch.Generator().manual_seed(4)
    x = torch.randn(8, H, generator=g)
    x[1] *= 1e6
    x[2] *= 1e-6
    x[3, ::2] *= 1e-4
    x[4] = 0
    x[5, 7] = float("inf")
    x[6, 9] = float("nan")
    x = x.bfloat16()
    ids = torch.zeros(8, 1, dtype=torch.int32)
    gates = torch.ones(8, 1)
    y = nv.expert_mlp(x.cuda(), up, down, ids.cuda(), gates.cuda()).cpu().double()
    want, bound = reference(x, up_v, down_v, ids, gates, block, None if up.amax is None else up.amax.cpu())
    fine = [0, 1, 2, 3, 4, 7]
    assert bool(((y - want).abs() <= bound)[fine].all())
    assert bool((y[4] == 0).all())
    assert not bool(torch.isfinite(y[5:7]).any())


@pytest.mark.parametrize("block", [16, 32])
def test_range_of_one_or_two_tokens(block):
    E, H, F = 3, 512, 96
    up, up_v = stack(E, 2 * F, H, block, 1, H ** -0.5)
    down, down_v = stack(E, H, F, block, 2, F ** -0.5)
    amax = None if up.amax is None else up.amax.cpu()
    ids = torch.tensor([[0, 2], [1, 0]], dtype=torch.int32)
    gates = torch.tensor([[0.5, 0.25], [1.0, 2.0]])
    for scale, at, value in ((1e6, 0, None), (1e-6, 0, None), (1.0, 7, float("inf")), (1.0, 500, float("nan"))):
        x = torch.randn(2, H, generator=torch.Generator().manual_seed(5)) * torch.tensor([[scale], [1.0]])
        if value is not None:
            x[0, at] = value
        x = x.bfloat16()
        for T in (1, 2):
            y = nv.expert_mlp(x[:T].cuda(), up, down, ids[:T].cuda(), gates[:T].cuda()).cpu().double()
            want, bound = reference(x[:T], up_v, down_v, ids[:T], gates[:T], block, amax)
            first = 0 if value is None else 1
            assert bool(((y - want).abs() <= bound)[first:].all())
            assert value is None or not bool(torch.isfinite(y[0]).any())


def test_empty_sizes():
    """No inner or no hidden columns: zeros, or nothing."""
    def op(n, k):
        return nv.FP4Operand(torch.zeros(2, n, k // 2, dtype=torch.uint8, device="cuda"),
                             torch.zeros(2, n, k // 32, dtype=torch.uint8, device="cuda"), None, 32)
    for T in (1, 5):
        ids, gates = torch.zeros(T, 1, dtype=torch.int32, device="cuda"), torch.ones(T, 1, device="cuda")
        y = nv.expert_mlp(torch.ones(T, 64, device="cuda").bfloat16(), op(0, 64), op(64, 0), ids, gates)
        assert y.shape == (T, 64) and bool((y == 0).all())
        y = nv.expert_mlp(torch.ones(T, 0, device="cuda").bfloat16(), op(64, 0), op(0, 32), ids, gates)
        assert y.shape == (T, 0)
