"""4-bit operators past 32-bit offsets: the same results as for the part alone."""
import pytest
import torch

import nvfp4_block_scaled_amax_gb300 as nv

pytestmark = [pytest.mark.gpu, pytest.mark.slow]


def random_operand(rows, k, seed, block=16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return nv.FP4Operand(torch.randint(0, 256, (rows, k // 2), generator=g, device="cuda", dtype=torch.uint8),
                         torch.randint(0x30, 0x40, (rows, k // block), generator=g, device="cuda", dtype=torch.uint8),
                         torch.full((1,), 2688.0, device="cuda") if block == 16 else None, block)


def rows_of(q, at):
    return nv.FP4Operand(q.data[at].contiguous(), q.scale[at].contiguous(), q.amax, q.block)


@pytest.mark.parametrize("m", [7, 300])
def test_weights_past_4_gib(m):
    n, k = 270336, 32768                       # 4.4e9 bytes of codes
    a, b = random_operand(m, k, 1), random_operand(n, k, 2)
    y = nv.matmul_fp4(a, b)
    for at in (slice(0, 256), slice(131072, 131072 + 512), slice(n - 384, n)):
        assert torch.equal(y[:, at], nv.matmul_fp4(a, rows_of(b, at)))


def test_output_past_2_31_elements():
    m, n, k = 33000, 66100, 64                 # rows off 16-byte boundaries in BF16 for odd n: n % 8 = 4
    a, b = random_operand(m, k, 3, 32), random_operand(n, k, 4, 32)
    y = nv.matmul_fp4(a, b)
    for at in (slice(0, 128), slice(m - 300, m)):
        assert torch.equal(y[at], nv.matmul_fp4(rows_of(a, at), b))


def test_cast_past_2_32_elements():
    m, n = 131328, 32896
    x = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    for at in range(0, m, 16416):
        x[at:at + 16416] = torch.randn(min(16416, m - at), n, generator=g, device="cuda").bfloat16()
    q = nv.quantize_mxfp4(x, colwise=True, swizzled=True)
    tail = nv.quantize_mxfp4(x[-256:].contiguous(), colwise=True, swizzled=True)
    assert torch.equal(q.row.data[-256:], tail.row.data)
    assert torch.equal(q.row.scale[-256 * (n // 32):], tail.row.scale)
    assert torch.equal(q.col.data[:, -128:], tail.col.data)
    back = nv.dequantize_fp4(q.row)
    assert torch.equal(back[-256:], nv.dequantize_fp4(tail.row))


@pytest.mark.parametrize("T", [1, 5])
def test_layer_past_4_gib(T):
    E, H, F = 44, 10240, 10240                 # 4.6e9 bytes of gate and up codes
    stack = lambda n, k, seed: nv.FP4Operand(*(lambda q: (q.data.view(E, n, k // 2), q.scale.view(E, n, k // 16),  # noqa: E731
                                                          torch.full((E,), 30.0, device="cuda")))(random_operand(E * n, k, seed)))
    up, down = stack(2 * F, H, 1), stack(H, F, 2)
    one = lambda q, e: nv.FP4Operand(q.data[e:e + 1], q.scale[e:e + 1], q.amax[e:e + 1])  # noqa: E731
    x = torch.randn(T, H, device="cuda").bfloat16()
    gates = torch.ones(T, 1, device="cuda")
    for e in (0, 21, E - 1):
        ids = torch.full((T, 1), e, dtype=torch.int32, device="cuda")
        y = nv.expert_mlp(x, up, down, ids, gates)
        assert bool(torch.isfinite(y).all())
        # the same sums, but a cluster may share them otherwise: a few units of FP32 of the magnitudes, before one rounding
        want = nv.expert_mlp(x, one(up, e), one(down, e), torch.zeros_like(ids), gates)
        assert float((y.double() - want.double()).norm() / want.double().norm()) < 2.0 ** -8
