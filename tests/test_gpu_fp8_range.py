"""Products whose scales are small or large together: the product of two scales leaves FP32's normal range, the result
does not.  The number of rows picks the kernel, so every size here goes through the same checks."""
import pytest
import torch

import nvfp4_block_scaled_amax_gb300 as nv

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
BLOCK = 128
SIZES = [(3, 200, 400), (40, 264, 1040), (700, 640, 656), (1500, 1300, 400)]  # few rows, and whole 256 x 256 tiles


def blocks(n):
    return -(-n // BLOCK)


def operand(rows, cols, block_rows, seed, values, exponents, lead=()):
    """Codes drawn from `values`, scales 2^e for e drawn from the range `exponents`; fractions of any bits."""
    g = torch.Generator().manual_seed(seed)
    pick = torch.randint(0, len(values), (*lead, rows, cols), generator=g)
    codes = torch.tensor(values)[pick].to(torch.float8_e4m3fn)
    shape = (*lead, blocks(cols), rows) if block_rows == 1 else (*lead, blocks(rows), blocks(cols))
    scale = torch.exp2(exponents[0] + (exponents[1] - exponents[0]) * torch.rand(shape, generator=g).double()).float()
    return nv.FP8Operand(codes.cuda(), scale.cuda(), block_rows)


def exact(op):
    d, s = op.data.cpu().float().double(), op.scale.cpu().double()
    rows, cols = d.shape[-2:]
    s = s.transpose(-1, -2) if op.block_rows == 1 else s.repeat_interleave(BLOCK, -2)[..., :rows, :]
    return d * s.repeat_interleave(BLOCK, -1)[..., :cols]


def check(got, a, b):
    """128 terms of a block with at most a unit each (the tensor cores may truncate), a block's two scales and its sum
    with three roundings more, each of at most a unit or the smallest normal number's unit."""
    want, size = a @ b.t(), a.abs() @ b.abs().t()
    steps = 128 + blocks(a.shape[1]) + 4
    bound = steps * 2 * U32 * size + steps * 2.0 ** -149
    assert bool(torch.isfinite(got).all())
    assert bool(((got.cpu().double() - want).abs() <= bound).all())


FULL = [0.0, 1.0, -1.5, 448.0, -104.0, 0.0625, 13.0]
TINY = [0.0] * 24 + [2.0 ** -9, -(2.0 ** -9), 2.0 ** -8]  # one in nine; products of 2^-18 to 2^-16


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("values,ea,eb", [(FULL, (-72, -68), (-72, -68)),   # scale products near 2^-140: subnormal
                                          (FULL, (-100, -96), (-30, -2)),   # normal for some blocks only
                                          (TINY, (66, 68), (66, 68)),       # near 2^134: infinite, the sums far below 1
                                          (FULL, (96, 100), (-100, -60))])  # normal, far apart
def test_scales_far_from_one(values, ea, eb, M, N, K, block_rows):
    a, b = operand(M, K, 1, M, values, ea), operand(N, K, block_rows, N, values, eb)
    got = nv.matmul_fp8(a, b, out_dtype=torch.float32)
    check(got, exact(a), exact(b))
    assert nv.device_status() == 0


def test_scales_far_from_one_by_expert():
    counts = [0, 700, 3, 300, 41]
    off = [0, 0, 700, 703, 1003, 1044]
    N, K = 520, 656
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    for rows in (off[-1], 5):  # whole tiles, and the kernel for few rows
        a = operand(rows, K, 1, 1, FULL, (-72, -68))
        b = operand(N, K, 128, 2, FULL, (-72, -68), lead=(len(counts),))
        got = nv.matmul_fp8_grouped(a, b, offsets.clamp(max=rows), out_dtype=torch.float32)
        av, bv = exact(a), exact(b)
        for e in range(len(counts)):
            r = slice(min(off[e], rows), min(off[e + 1], rows))
            check(got[r], av[r], bv[e])


@pytest.mark.parametrize("M,N,K", [(5, 256, 400), (700, 640, 656)])
def test_rows_do_not_depend_on_their_neighbours(M, N, K):
    """A row next to one whose scales are far off has the same bits as without it; zero and non-finite scales are what
    their products say."""
    a, b = operand(M, K, 1, 1, FULL, (-6, -2)), operand(N, K, 128, 2, FULL, (-6, -2))
    want = nv.matmul_fp8(a, b, out_dtype=torch.float32)
    scale = a.scale.clone()
    scale[:, 1] = 0.0
    scale[0, 2] = 2.0 ** -140
    scale[0, 3], scale[0, 4] = float("inf"), float("nan")
    got = nv.matmul_fp8(nv.FP8Operand(a.data, scale), b, out_dtype=torch.float32)
    others = [r for r in range(M) if r not in (1, 2, 3, 4)]
    assert torch.equal(got[others], want[others])
    assert bool((got[1] == 0).all()) and bool(torch.isnan(got[4]).all()) and not bool(torch.isfinite(got[3]).any())
    check(got[2:3], exact(nv.FP8Operand(a.data, scale))[2:3], exact(b))
