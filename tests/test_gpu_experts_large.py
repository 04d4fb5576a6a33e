"""Sizes whose byte or element offsets pass 32 bits: the last rows come out right."""
import pytest
import torch

import nvfp4_block_scaled_amax_gb300 as nv

pytestmark = [pytest.mark.gpu, pytest.mark.slow]

U32, U16 = 2.0 ** -24, 2.0 ** -8  # half a unit in the last place, relative: FP32, BF16


def codes(rows, cols, seed, lead=()):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = torch.randint(0, 256, (*lead, rows, cols), generator=g, device="cuda", dtype=torch.uint8)
    return torch.where((c & 127) == 127, torch.zeros_like(c), c).view(torch.float8_e4m3fn)


def scales(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.exp2(4 * torch.rand(shape, generator=g, device="cuda") - 8)


def check(got, a, b):
    """As the smaller products: 128 terms and the blocks in FP32, one rounding to BF16."""
    want, size = a @ b.t(), a.abs() @ b.abs().t()
    bound = (128 + a.shape[1] // 128 + 4) * 2 * U32 * size * (1 + U16) + U16 * want.abs()
    assert bool(((got.double() - want).abs() <= bound).all())


def test_product_with_more_than_two_to_the_31_outputs():
    M, N, K = 66000, 33000, 128  # 2.18e9 outputs
    a, b = nv.FP8Operand(codes(M, K, 1), scales((1, M), 2)), nv.FP8Operand(codes(N, K, 3), scales((1, N), 4))
    y = nv.matmul_fp8(a, b)
    av = a.data[-300:].double() * a.scale[0, -300:, None].double()
    bv = b.data.double() * b.scale[0, :, None].double()
    check(y[-300:], av, bv)
    av = a.data[32700:32800].double() * a.scale[0, 32700:32800, None].double()
    check(y[32700:32800], av, bv)


def test_experts_whose_weights_pass_two_to_the_31_bytes():
    E, N, K, rows = 17, 8192, 16384, 40  # 2.28e9 bytes of weights
    b = nv.FP8Operand(codes(N, K, 1, lead=(E,)), scales((E, N // 128, K // 128), 2), block_rows=128)
    offsets = torch.tensor([0] * 16 + [9, rows], dtype=torch.int32, device="cuda")  # the last two experts
    a = nv.FP8Operand(codes(rows, K, 3), scales((K // 128, rows), 4))
    y = nv.matmul_fp8_grouped(a, b, offsets)
    av = a.data.double() * a.scale.t().double().repeat_interleave(128, 1)
    for e, r in ((15, slice(0, 9)), (16, slice(9, rows))):
        bv = b.data[e].double() * b.scale[e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
        check(y[r], av[r], bv)


def test_cast_of_more_than_two_to_the_31_elements():
    M, N = 65552, 33024  # 2.16e9 elements
    x = torch.empty(M, N, device="cuda", dtype=torch.bfloat16).normal_()
    q = nv.quantize_fp8(x, colwise=True)
    for part, op in ((x[-200:], q.row.data[-200:]), (x[:, -200:].t(), q.col.data[-200:])):
        v = torch.nn.functional.pad(part.float(), (0, -part.shape[1] % 128)).view(200, -1, 128)
        factor = torch.full((), 448.0, device="cuda") / v.abs().amax(-1).clamp(min=2.0 ** -100)
        want = (v * factor[..., None]).flatten(1)[:, :part.shape[1]].clamp(-448, 448).to(torch.float8_e4m3fn)
        assert torch.equal(op.view(torch.uint8), want.view(torch.uint8))


def test_rows_of_more_than_two_to_the_31_elements():
    T, topk, E, H = 33000, 2, 16, 33280  # 2.2e9 elements of rows
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randint(0, E, (T, topk), generator=g, device="cuda", dtype=torch.int32)
    x = torch.empty(T, H, device="cuda", dtype=torch.bfloat16).normal_()
    rows, plan = nv.dispatch_tokens(x, ids, E)
    slot = plan.slot_of_row.long()
    for part in (slice(0, 64), slice(T - 32, T + 32), slice(2 * T - 64, 2 * T)):
        assert torch.equal(rows[part], x[slot[part] // topk])
    y = nv.combine_tokens(rows, plan)
    for part in (slice(0, 64), slice(T - 64, T)):
        assert torch.equal(y[part], (x[part].float() * 2).bfloat16())  # each token is there twice
    drows, dw = nv.combine_tokens_grad(y, rows, plan)
    assert torch.equal(drows[-64:], y[slot[-64:] // topk])
    assert dw.shape == (T, topk)


@pytest.mark.parametrize("M,N", [(1, 524288), (20, 524160)])
def test_few_rows_through_a_very_wide_matrix(M, N):
    """4096 (and 4095) tiles of weights: tile indexes times 2^20 would pass 32 bits."""
    K = 144
    a, b = nv.FP8Operand(codes(M, K, 1), scales((2, M), 2)), nv.FP8Operand(codes(N, K, 3), scales((2, N), 4))
    y = nv.matmul_fp8(a, b, out_dtype=torch.float32)
    av = a.data.double() * a.scale.t().double().repeat_interleave(128, 1)[:, :K]
    bv = b.data.double() * b.scale.t().double().repeat_interleave(128, 1)[:, :K]
    check(y, av, bv)


def test_sort_whose_member_and_alignment_pass_two_to_the_31_together():
    align = 1000003
    T = 2147 * align  # already a multiple: a member of T rows, although T + align - 1 > 2^31
    ids = torch.zeros(T, 1, device="cuda", dtype=torch.int32)
    plan = nv.sort_tokens(ids, 1, align=align)
    assert plan.offsets.tolist() == [0, T] and plan.rows == T
    for s in range(0, T, 1 << 28):
        e = min(s + (1 << 28), T)
        want = torch.arange(s, e, device="cuda", dtype=torch.int32)
        assert torch.equal(plan.row_of_slot[s:e, 0], want) and torch.equal(plan.slot_of_row[s:e], want)
