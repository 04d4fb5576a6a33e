"""Member offsets that a product by expert does not take: reported by the status word, nothing written outside the
output, and every well-formed member as it should be."""
import pytest
import torch

import nvfp4_block_scaled_amax_gb300 as nv

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
BLOCK = 128
BAD_OFFSETS = 4
FOREIGN = 7.0


def blocks(n):
    return -(-n // BLOCK)


def operand(rows, cols, block_rows, seed, lead=()):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (*lead, rows, cols), generator=g, dtype=torch.int32).to(torch.uint8)
    codes = torch.where((codes & 127) == 127, torch.zeros_like(codes), codes)
    shape = (blocks(cols), rows) if block_rows == 1 else (blocks(rows), blocks(cols))
    scale = torch.exp2(4 * torch.rand(*lead, *shape, generator=g) - 8)
    return nv.FP8Operand(codes.cuda().view(torch.float8_e4m3fn), scale.cuda(), block_rows)


def exact(op):
    d, s = op.data.cpu().float().double(), op.scale.cpu().double()
    rows, cols = d.shape[-2:]
    s = s.transpose(-1, -2) if op.block_rows == 1 else s.repeat_interleave(BLOCK, -2)[..., :rows, :]
    return d * s.repeat_interleave(BLOCK, -1)[..., :cols]


def check(got, a, b):
    """128 terms of a block with at most a unit each, three roundings for each block."""
    want, size = a @ b.t(), a.abs() @ b.abs().t()
    bound = (128 + blocks(a.shape[1]) + 4) * 2 * U32 * size
    assert bool(((got.cpu().double() - want).abs() <= bound).all())


def guarded(*shape):
    """(storage, the output in the middle of it)"""
    n, edge = 1, 256 * shape[-1]
    for d in shape:
        n *= d
    storage = torch.full((n + 2 * edge,), FOREIGN, device="cuda")
    return storage, storage[edge:edge + n].view(shape)


def check_outside(storage, out):
    edge = (storage.numel() - out.numel()) // 2
    assert bool((storage[:edge] == FOREIGN).all()) and bool((storage[edge + out.numel():] == FOREIGN).all())


def as_taken(offsets, rows):
    """Each at least the one before, all inside the rows."""
    taken = [min(max(offsets[0], 0), rows)]
    for v in offsets[1:]:
        taken.append(max(taken[-1], min(max(v, 0), rows)))
    return taken


# few rows a member (the kernel for few rows), and members of whole tiles
@pytest.mark.parametrize("offsets,rows", [([0, 40, 20, 60, 50], 60), ([0, 10, 500, 600, 30], 60), ([0, -5, 9, 12, 60], 60),
                                          ([4, 10, 20, 30, 60], 60), ([-(2 ** 31), 2 ** 31 - 1, -1, 2 ** 31 - 1, 7], 60),
                                          ([0, 900, 500, 1500, 1400], 1500), ([0, 700, 5000, 6000, 100], 1500),
                                          ([-9, 700, -3, 1100, 1500], 1500), ([0, 1500, 0, 1500, 0], 1500)])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_product(offsets, rows, block_rows):
    N, K, E = 300, 272, len(offsets) - 1
    a, b = operand(rows, K, 1, rows), operand(N, K, block_rows, N, lead=(E,))
    storage, out = guarded(rows, N)
    assert nv.device_status() == 0
    nv.matmul_fp8_grouped(a, b, torch.tensor(offsets, dtype=torch.int32, device="cuda"), out=out)
    assert nv.device_status() == BAD_OFFSETS and nv.device_status() == 0
    check_outside(storage, out)
    av, bv, off = exact(a), exact(b), as_taken(offsets, rows)
    assert bool((out[:off[0]] == FOREIGN).all()) and bool((out[off[-1]:] == 0).all())
    for e in range(E):
        check(out[off[e]:off[e + 1]], av[off[e]:off[e + 1]], bv[e])
    # and the same call with offsets that it takes
    nv.matmul_fp8_grouped(a, b, torch.tensor([0, *off[1:]], dtype=torch.int32, device="cuda"), out=out)
    assert nv.device_status() == 0


@pytest.mark.parametrize("offsets,rows", [([0, 100, 256, 512], 512), ([0, 128, 64, 512], 512), ([0, 640, 128, 512], 512),
                                          ([-128, 128, 256, 512], 512), ([0, 128, 256, 600], 512)])
@pytest.mark.parametrize("M,N", [(40, 200), (520, 776)])
def test_weight_gradient(offsets, rows, M, N):
    a, b = operand(M, rows, 1, M), operand(N, rows, 1, N)
    storage, out = guarded(len(offsets) - 1, M, N)
    assert nv.device_status() == 0
    nv.matmul_fp8_grouped_wgrad(a, b, torch.tensor(offsets, dtype=torch.int32, device="cuda"), out=out)
    assert nv.device_status() == BAD_OFFSETS and nv.device_status() == 0
    check_outside(storage, out)
    av, bv, off = exact(a), exact(b), as_taken(offsets, rows)
    for e in range(len(offsets) - 1):
        # a block that a member shares counts whole
        r = slice(off[e] // BLOCK * BLOCK, min(blocks(off[e + 1]) * BLOCK, rows)) if off[e] < off[e + 1] else slice(0, 0)
        check(out[e], av[:, r], bv[:, r])


def test_a_plan_for_members_of_one_row_is_reported():
    """The offsets of tokens sorted without padding: no weight gradient can be made of them in blocks of 128 tokens."""
    ids = (torch.arange(150, device="cuda", dtype=torch.int32) % 3).view(150, 1)
    x = torch.randn(150, 128, device="cuda", dtype=torch.bfloat16)
    for align, status in ((1, BAD_OFFSETS), (128, 0)):
        rows, plan = nv.dispatch_tokens(x, ids, 3, align=align)
        rows = torch.nn.functional.pad(rows, (0, 0, 0, -rows.shape[0] % 16))
        q = nv.quantize_fp8(rows, rowwise=False, colwise=True)
        nv.matmul_fp8_grouped_wgrad(q.col, q.col, plan.offsets)
        assert nv.device_status() == status


@pytest.mark.parametrize("M,N", [(40, 200), (520, 776)])
def test_a_last_member_may_end_with_the_rows(M, N):
    rows, off = 304, [0, 128, 128, 304]
    a, b = operand(M, rows, 1, M), operand(N, rows, 1, N)
    got = nv.matmul_fp8_grouped_wgrad(a, b, torch.tensor(off, dtype=torch.int32, device="cuda"))
    av, bv = exact(a), exact(b)
    for e in range(3):
        check(got[e], av[:, off[e]:off[e + 1]], bv[:, off[e]:off[e + 1]])
    assert nv.device_status() == 0
