"""The MXFP4 cast, its reading back, and the product of 4-bit operands, against 64-bit arithmetic."""
import pytest
import torch

import nvfp4_block_scaled_amax_gb300 as nv
from fp4_testutil import mx_cast, operand, pack, random_parts, swizzle, values

pytestmark = pytest.mark.gpu

U32, U16 = 2.0 ** -24, 2.0 ** -8


def tensor(M, N, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, N, generator=g)
    x = torch.where(torch.rand(M, N, generator=g) < 0.01, x * 50, x)
    if M >= 64 and N >= 64:
        x[7] = 0.0                                      # rows and columns of zeros
        x[:, 33] = 0.0
        x[16, :32] = 1e-38 * torch.arange(32)           # subnormal scales
        x[17, :32] = 2.0 ** -140
        x[40, :32] = 3e38 / 40 * torch.arange(32)       # the largest scales
        x[33, ::3] = 2.0 ** torch.arange(0, N, 3).remainder(20).float()
        x[41, 5], x[42, 6], x[43, 40] = float("inf"), float("-inf"), float("nan")
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(1, 32), (7, 4096), (32, 32), (64, 96), (96, 1056), (128, 128), (160, 288), (256, 640),
                                   (77, 160)])
def test_mxfp4_cast(shape, dtype):
    M, N = shape
    x = tensor(M, N, 1, dtype)
    colwise = M % 32 == 0
    for row, col in ((True, False), (True, colwise), (not colwise, colwise)):
        for swizzled in (False, True) if M % 128 == 0 and N % 128 == 0 else (False,):
            q = nv.quantize_mxfp4(x.cuda(), rowwise=row, colwise=col, swizzled=swizzled)
            assert (q.row is not None) == row and (q.col is not None) == col
            for op, ref in ((q.row, x), (q.col, x.t())):
                if op is None:
                    continue
                code, byte = mx_cast(ref)
                assert torch.equal(op.scale.cpu(), swizzle(byte) if swizzled else byte.reshape(-1))
                assert torch.equal(op.data.cpu(), pack(code))
                for out in (torch.bfloat16, torch.float32):
                    got = nv.dequantize_fp4(op, out).cpu()
                    want = values(pack(code), byte, None, 32)
                    assert torch.equal(got.double().nan_to_num(nan=-1.0), want.nan_to_num(nan=-1.0))
    assert nv.device_status() == 0


def test_mxfp4_cast_of_every_bf16_value():
    """Each BF16 number in a block that it leads: ties, subnormals and the largest numbers."""
    bits = torch.arange(1 << 15, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = bits[:, None].float() * torch.tensor([1.0, -1.0, 0.75, 0.5] + [0.125 * i for i in range(28)])
    x = x.to(torch.bfloat16)
    q = nv.quantize_mxfp4(x.cuda()).row
    code, byte = mx_cast(x)
    assert torch.equal(q.scale.cpu(), byte.reshape(-1))
    assert torch.equal(q.data.cpu(), pack(code))
    # as columns: neighbouring blocks of every size, beside ones that are not finite
    for shuffled in (False, True):
        y = x[torch.randperm(len(x), generator=torch.Generator().manual_seed(1))] if shuffled else x
        q = nv.quantize_mxfp4(y.t().contiguous().cuda(), colwise=True)
        for op, ref in ((q.row, y.t()), (q.col, y)):
            code, byte = mx_cast(ref)
            assert torch.equal(op.scale.cpu(), byte.reshape(-1))
            assert torch.equal(op.data.cpu(), pack(code))


def test_nvfp4_reading_back_is_dequantize():
    x = tensor(256, 384, 5, torch.float32).nan_to_num(0.0, 1.0, 1.0).clamp(-100, 100).cuda()
    for mode, sw in (("1d", False), ("2d", True), ("row_scaled", False)):
        t = nv.quantize(x, mode, swizzled=sw)
        want = nv.dequantize(t.data_row, t.scale_row, t.amax_row, swizzled=sw, row_scaled=mode == "row_scaled")
        assert torch.equal(nv.dequantize_fp4(t.row), want)
        if t.data_col is not None:
            assert torch.equal(nv.dequantize_fp4(t.col), nv.dequantize(t.data_col, t.scale_col, t.amax_col, swizzled=sw))


def check_product(m, n, k, block, per_row, a_sw, b_sw, out_dtype, exact, seed=0):
    pa = random_parts(m, k, block, 2 * seed + 1, exact, per_row)
    pb = random_parts(n, k, block, 2 * seed + 2, exact, per_row and n % 2 == 0)
    y = nv.matmul_fp4(operand(pa, block, a_sw), operand(pb, block, b_sw), out_dtype=out_dtype)
    assert y.shape == (m, n) and y.dtype == out_dtype
    a, b = values(*pa, block).cuda(), values(*pb, block).cuda()
    want = a @ b.t()
    if exact:
        assert torch.equal(y.double(), want.to(out_dtype).double())
    else:
        # K products summed in 32 bits in some order, three more roundings (the factors, their product, the result's)
        tol = ((k + 4) * U32) * (a.abs() @ b.abs().t()) + (U16 if out_dtype == torch.bfloat16 else 0.0) * want.abs()
        assert bool(((y.double() - want).abs() <= tol * 1.001).all())
    assert nv.device_status() == 0


SHAPES = [(1, 128, 256), (1, 1, 32), (3, 5, 64), (7, 9, 96), (16, 256, 512), (17, 200, 160), (33, 129, 288),
          (64, 128, 4096), (1, 640, 4096), (100, 300, 2080), (128, 128, 128), (128, 256, 384), (130, 70, 32),
          (256, 384, 640), (333, 1091, 2080), (384, 520, 1184), (512, 512, 1024)]


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("shape", SHAPES)
def test_product(shape, block):
    m, n, k = shape
    for a_sw in (False, True):
        for b_sw in (False, True):
            if (a_sw and (m % 128 or k % 128)) or (b_sw and (n % 128 or k % 128)):
                continue
            for out_dtype in (torch.bfloat16, torch.float32):
                check_product(m, n, k, block, False, a_sw, b_sw, out_dtype, True)
                check_product(m, n, k, block, block == 16, a_sw, b_sw, out_dtype, False, 1)


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("shape", [(64, 130, 16416), (16, 128, 16416), (50, 5000, 8224), (120, 20000, 1056),
                                   (1500, 2500, 1312), (128, 40064, 640), (5000, 4100, 96), (2560, 4864, 1408),
                                   (4096, 4352, 256), (65, 257, 4128)])
def test_product_long(shape, block):
    """More stages than shared memory holds, and more tiles than CTAs, with scales of both layouts."""
    m, n, k = shape
    check_product(m, n, k, block, False, False, False, torch.float32, True)
    if n % 128 == 0 and k % 128 == 0:
        check_product(m, n, k, block, False, m % 128 == 0, True, torch.bfloat16, True)


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("shape", [(640, 1280, 2048), (1300, 2600, 1536), (1300, 2600, 1280), (2304, 4480, 512),
                                   (70, 9000, 1792), (1111, 2222, 2592)])
def test_product_compact(shape, block):
    """Compact scales of either side or both, read two stages at a time: rows that are whole pairs of stages, whole
    stages, and neither; odd numbers of stages; many tiles."""
    m, n, k = shape
    for a_sw in (False, True) if m % 128 == 0 and k % 128 == 0 else (False,):
        for b_sw in (False, True) if n % 128 == 0 and k % 128 == 0 else (False,):
            check_product(m, n, k, block, block == 16, a_sw, b_sw, torch.float32, True)
            check_product(m, n, k, block, False, a_sw, b_sw, torch.bfloat16, True, 3)


def test_product_of_nothing():
    for block in (16, 32):
        for m, n, k in ((0, 5, 64), (5, 0, 64), (5, 7, 0)):
            a = operand(random_parts(m, k, block, 1, True), block)
            b = operand(random_parts(n, k, block, 2, True), block)
            y = nv.matmul_fp4(a, b)
            assert y.shape == (m, n) and bool((y == 0).all())
