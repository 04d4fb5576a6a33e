"""The E4M3 cast with a scale for each block of 128, and the product of such operands, against 64-bit arithmetic."""
import pytest
import torch

import nvfp4_block_scaled_amax_gb300 as nv

pytestmark = pytest.mark.gpu

U32, U16 = 2.0 ** -24, 2.0 ** -8
BLOCK = 128


def blocks(n):
    return -(-n // BLOCK)


def e4m3(v):
    """Nearest E4M3 value of a 64-bit tensor: ties to even, at most 448."""
    a = v.abs().clamp(max=448.0)
    step = torch.ldexp(torch.ones_like(a), torch.frexp(a).exponent.clamp(min=-5) - 4)
    return torch.copysign(torch.round(a / step) * step, v)


def block_amax(x, block_rows):
    """max|x| of each element's block, in 64 bits, for one matrix."""
    M, N = x.shape
    p = torch.nn.functional.pad(x.abs(), (0, blocks(N) * BLOCK - N, 0, blocks(M) * BLOCK - M))
    if block_rows == 1:
        a = p.view(p.shape[0], -1, BLOCK).amax(-1)
        return a[:M], a.repeat_interleave(BLOCK, 1)[:M, :N]
    a = p.view(blocks(M), BLOCK, -1, BLOCK).amax((1, 3))
    return a, a.repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)[:M, :N]


def check_cast(x, q, block_rows):
    """q: the operand of the matrix x (64 bits, exact).  s and r are one rounding from a/448 and 448/a, x * r another,
    so each code is the rounding of some value within 3 units of the exact quotient."""
    amax, per = block_amax(x, block_rows)
    amax, per = amax.clamp(min=2.0 ** -100), per.clamp(min=2.0 ** -100)
    s = q.scale.cpu().double()
    s = s.t() if block_rows == 1 else s
    fine = torch.isfinite(amax)
    assert bool((s[~fine] == float("inf")).all())
    assert bool(((s - amax / 448).abs() <= U32 * amax / 448 * 1.01)[fine].all())
    codes = q.data.cpu().float().double()
    exact = x * (448 / per)
    lo, hi = e4m3(exact * (1 - 3 * U32)), e4m3(exact * (1 + 3 * U32))
    right = (codes >= torch.minimum(lo, hi)) & (codes <= torch.maximum(lo, hi))
    # a block with an infinity: NaN for the infinity itself, zero (x * 0) for the others
    right = torch.where(torch.isfinite(per), right, torch.where(torch.isfinite(x), codes == 0, torch.isnan(codes)))
    assert bool(right.all())


def values(M, N, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, N, generator=g)
    x = torch.where(torch.rand(M, N, generator=g) < 0.01, x * 50, x)
    if M > 40 and N > 140:
        x[7] = 0.0                                     # a row of zeros
        x[:, 130] = 0.0                                # a column of zeros
        x[16, :128] = 1e-38 * torch.arange(128)        # below the floor
        x[33, :] = torch.arange(N) / 448.0 * 3e38 / N  # large, and infinite from element 508 on
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("shape", [(1, 16), (1, 4096), (16, 16), (77, 1040), (128, 128), (144, 272), (208, 2064),
                                   (3, 48, 176), (2, 160, 144)])
def test_cast(shape, block_rows, dtype):
    lead, (M, N) = shape[:-2], shape[-2:]
    x = torch.stack([values(M, N, s, dtype) for s in range(lead[0] if lead else 1)])
    x = x if lead else x[0]
    colwise = M % 16 == 0
    for rowwise, col in ((True, False), (True, colwise), (not colwise, colwise)):
        q = nv.quantize_fp8(x.cuda(), block_rows=block_rows, rowwise=rowwise, colwise=col)
        assert (q.row is not None) == rowwise and (q.col is not None) == col
        parts = x.double().reshape(-1, M, N)
        for i, part in enumerate(parts):
            for op, ref in ((q.row, part), (q.col, part.t())):
                if op is not None:
                    one = nv.FP8Operand(op.data.reshape(-1, *op.data.shape[-2:])[i],
                                        op.scale.reshape(-1, *op.scale.shape[-2:])[i], block_rows)
                    check_cast(ref, one, block_rows)


def test_cast_is_the_plain_formula_bit_for_bit():
    x = values(256, 512, 3, torch.float32).cuda()
    q = nv.quantize_fp8(x, colwise=True)
    for op, src in ((q.row, x), (q.col, x.t().contiguous())):
        v = src.view(src.shape[0], -1, BLOCK)
        amax = v.abs().amax(-1).clamp(min=2.0 ** -100)
        top = torch.full((), 448.0, device="cuda")
        assert torch.equal(op.scale.t(), amax / top)
        want = (v * (top / amax)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(src.shape)
        assert torch.equal(op.data.view(torch.uint8), want.view(torch.uint8))


def test_cast_keeps_non_finite_values_visible():
    x = torch.ones(32, 256, device="cuda")
    x[3, 5], x[9, 200] = float("inf"), float("nan")
    q = nv.quantize_fp8(x, colwise=True)
    back = q.row.dequantize().cpu()
    assert bool(torch.isnan(back[3, :128]).all()) and bool((back[3, 128:] == 1).all())
    assert bool(torch.isnan(back[9, 200])) and int(torch.isnan(back).sum()) == 129
    assert bool(torch.isnan(q.col.dequantize().cpu()[5]).all())
    y = nv.matmul_fp8(q.row, q.row, out_dtype=torch.float32).cpu()
    assert bool(torch.isnan(y[3]).all()) and bool(torch.isnan(y[9]).all())
    assert int(torch.isnan(y).sum()) == 4 * 32 - 4


def test_cast_sizes_of_zero():
    q = nv.quantize_fp8(torch.zeros(0, 64, device="cuda"), colwise=True)
    assert q.row.data.shape == (0, 64) and q.col.data.shape == (64, 0) and q.col.scale.shape == (0, 64)


def operand(rows, cols, block_rows, seed, lead=()):
    """Random codes (all finite ones) and scales over several binades."""
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


def check_product(got, a, b, dtype):
    """A block's 128 exact products are added in FP32 with at most a unit each (the tensor cores may truncate), each
    block is scaled and added with three more roundings, the result is rounded once."""
    want, size = a @ b.t(), a.abs() @ b.abs().t()
    k = a.shape[1]
    out = U16 if dtype == torch.bfloat16 else 0.0
    bound = (128 + blocks(k) + 4) * 2 * U32 * size * (1 + out) + out * want.abs()
    worst = ((got.cpu().double() - want).abs() - bound).max() if got.numel() else 0.0
    assert float(worst) <= 0.0


SIZES = [(1, 1, 16), (1, 128, 128), (1, 5120, 4096), (3, 7, 144), (16, 257, 272), (17, 1000, 1040), (64, 512, 2048),
         (77, 131, 4112), (128, 128, 128), (129, 300, 384), (200, 2050, 1024), (333, 1091, 2064), (256, 256, 16),
         (700, 640, 656), (1500, 1300, 512), (2500, 2300, 272)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product(M, N, K, block_rows, dtype):
    a, b = operand(M, K, 1, M + K), operand(N, K, block_rows, N)
    got = nv.matmul_fp8(a, b, out_dtype=dtype)
    check_product(got, exact(a), exact(b), dtype)
    assert torch.equal(got, nv.matmul_fp8(a, b, out_dtype=dtype))  # the same bits every time
    assert nv.device_status() == 0


def test_product_writes_inside_its_output_only():
    M, N, K = 130, 259, 272
    a, b = operand(M, K, 1, 1), operand(N, K, 128, 2)
    for dtype in (torch.bfloat16, torch.float32):
        big = torch.full((M * N + 64,), 7.0, device="cuda", dtype=dtype)
        nv.matmul_fp8(a, b, out=big[:M * N].view(M, N))
        assert bool((big[M * N:] == 7).all())
        check_product(big[:M * N].view(M, N), exact(a), exact(b), dtype)


def test_product_sizes_of_zero():
    for M, N, K in ((0, 5, 32), (5, 0, 32), (5, 6, 0)):
        a, b = operand(M, K, 1, 1), operand(N, K, 128, 2)
        got = nv.matmul_fp8(a, b, out=torch.full((M, N), 3.0, device="cuda"))
        assert got.shape == (M, N) and bool((got == 0).all())


def member_offsets(counts, align=1):
    off = [0]
    for c in counts:
        off.append(off[-1] + -(-c // align) * align)
    return torch.tensor(off, dtype=torch.int32, device="cuda"), off


GROUPS = [([1], 128, 256), ([0, 3, 0, 5, 1, 0], 384, 272), ([130, 0, 1, 127, 128, 129], 200, 1040),
          ([16] * 9, 130, 528), ([900, 2, 0, 400], 264, 384), ([0, 0, 0], 64, 128), ([2] * 40, 512, 1024),
          ([33, 70, 64, 65, 0, 20], 136, 2048), ([1000, 300, 0, 1100, 513], 2200, 272)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("counts,N,K", GROUPS)
def test_grouped_product(counts, N, K, block_rows, dtype):
    E = len(counts)
    for align, spare in ((1, 0), (1, 3), (128, 200)):
        offsets, off = member_offsets(counts, align)
        R = off[-1] + spare
        if R == 0:
            continue
        a, b = operand(R, K, 1, R), operand(N, K, block_rows, N, lead=(E,))
        got = nv.matmul_fp8_grouped(a, b, offsets, out_dtype=dtype, out=torch.full((R, N), 9.0, device="cuda",
                                                                                  dtype=dtype))
        av, bv = exact(a), exact(b)
        for e in range(E):
            check_product(got[off[e]:off[e + 1]], av[off[e]:off[e + 1]], bv[e], dtype)
        assert bool((got[off[-1]:] == 0).all())
    assert nv.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts,M,N", [([1], 128, 256), ([0, 130, 0, 256], 200, 136), ([700, 128, 0, 300], 384, 520),
                                        ([0, 0], 64, 72), ([128] * 12, 136, 264), ([1500, 60], 264, 1000),
                                        ([300, 0, 520, 100], 1288, 1416)])
def test_weight_gradient(counts, M, N, dtype):
    offsets, off = member_offsets(counts, 128)
    for spare in (0, 144):
        R = off[-1] + spare
        a, b = operand(M, R, 1, M), operand(N, R, 1, N)
        got = nv.matmul_fp8_grouped_wgrad(a, b, offsets, out_dtype=dtype)
        av, bv = exact(a), exact(b)
        for e in range(len(counts)):
            check_product(got[e], av[:, off[e]:off[e + 1]], bv[:, off[e]:off[e + 1]], dtype)
            if counts[e] == 0:
                assert bool((got[e] == 0).all())
    assert nv.device_status() == 0


def integers(shape, seed, scale):
    """Multiples of `scale` with magnitudes 0..8 and one of 8 in every block: cast without any rounding when scale is
    a power of two times 448 / 8 ... so every code is exact."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(-7, 8, shape, generator=g).float()
    x[:, ::16] = 7.0
    x[::16] = 7.0
    return (x * scale).cuda()


def test_gradients_against_differences():
    """The three products of y = x w^T on inputs that the cast keeps exactly (7 * 2^6 = 448): every sum is an exact
    integer multiple, so the gradients must equal the differences of the loss <dy, y>."""
    M, N, K = 256, 128, 384
    x, w, dy = integers((M, K), 1, 64.0), integers((N, K), 2, 64.0), integers((M, N), 3, 64.0)
    qx, qw, qd = nv.quantize_fp8(x, colwise=True), nv.quantize_fp8(w, 128, colwise=True), nv.quantize_fp8(dy, colwise=True)
    f32 = torch.float32
    assert torch.equal(qx.row.dequantize(), x) and torch.equal(qw.col.dequantize(), w.t())
    dx, dw = nv.matmul_fp8(qd.row, qw.col, out_dtype=f32), nv.matmul_fp8(qd.col, qx.col, out_dtype=f32)

    def loss(xx, ww):
        y = nv.matmul_fp8(nv.quantize_fp8(xx).row, nv.quantize_fp8(ww, 128).row, out_dtype=f32)
        return float((y.double() * dy.double()).sum())
    base = loss(x, w)
    for i, j in ((0, 1), (13, 200), (255, 383)):
        step = torch.zeros_like(x)
        step[i, j] = -64.0 if float(x[i, j]) > 0 else 64.0
        assert loss(x + step, w) - base == float(dx[i, j]) * float(step[i, j])
    for i, j in ((0, 1), (77, 300), (127, 383)):
        step = torch.zeros_like(w)
        step[i, j] = -64.0 if float(w[i, j]) > 0 else 64.0
        assert loss(x, w + step) - base == float(dw[i, j]) * float(step[i, j])


def test_product_on_another_stream_and_in_a_graph():
    a, b = operand(200, 512, 1, 1), operand(300, 512, 128, 2)
    want = nv.matmul_fp8(a, b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = nv.matmul_fp8(a, b)
    s.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        again = nv.matmul_fp8(a, b)
    again.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, want)


def test_refusals():
    a, b = operand(8, 64, 1, 1), operand(8, 64, 128, 2)
    off = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    b3 = operand(8, 64, 128, 2, lead=(1,))
    x = torch.zeros(32, 64, device="cuda")
    for err, call in [
            (ValueError, lambda: nv.matmul_fp8(b, b)),                                     # a with 128-row blocks
            (ValueError, lambda: nv.matmul_fp8(a, operand(8, 48, 1, 1))),
            (ValueError, lambda: nv.matmul_fp8(a, b3)),
            (ValueError, lambda: nv.matmul_fp8(a, nv.FP8Operand(b.data, b.scale, 1))),     # scales of another layout
            (ValueError, lambda: nv.matmul_fp8(a, nv.FP8Operand(b.data, b.scale, 64))),
            (TypeError, lambda: nv.matmul_fp8(nv.FP8Operand(a.data.view(torch.uint8), a.scale), b)),
            (TypeError, lambda: nv.matmul_fp8(a, b, out_dtype=torch.float16)),
            (ValueError, lambda: nv.matmul_fp8(a, b, out=torch.zeros(8, 9, device="cuda"))),
            (ValueError, lambda: nv.matmul_fp8(nv.FP8Operand(a.data.cpu(), a.scale.cpu()), b)),
            (nv.NVFP4Error, lambda: nv.matmul_fp8(operand(8, 40, 1, 1), operand(8, 40, 1, 1))),  # K % 16
            (ValueError, lambda: nv.matmul_fp8_grouped(a, b, off)),
            (TypeError, lambda: nv.matmul_fp8_grouped(a, b3, off.long())),
            (ValueError, lambda: nv.matmul_fp8_grouped(a, b3, torch.tensor([0, 4, 8], dtype=torch.int32,
                                                                          device="cuda"))),
            (ValueError, lambda: nv.matmul_fp8_grouped_wgrad(a, b, off)),
            (TypeError, lambda: nv.quantize_fp8(x.half())),
            (ValueError, lambda: nv.quantize_fp8(x.t())),
            (ValueError, lambda: nv.quantize_fp8(x[0])),
            (nv.NVFP4Error, lambda: nv.quantize_fp8(x, block_rows=64)),
            (nv.NVFP4Error, lambda: nv.quantize_fp8(x, rowwise=False)),
            (nv.NVFP4Error, lambda: nv.quantize_fp8(x[:, :24].contiguous())),
            (nv.NVFP4Error, lambda: nv.quantize_fp8(x[:24], colwise=True))]:
        with pytest.raises(err):
            call()


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("M,N,K", [(3, 9900, 4112), (40, 9872, 4224),  # two CTAs share a tile's blocks
                                   (4700, 4500, 144)])                # more tiles per CTA than are worked out ahead
def test_product_of_many_tiles(M, N, K, block_rows):
    a, b = operand(M, K, 1, M + K), operand(N, K, block_rows, N)
    got = nv.matmul_fp8(a, b)
    check_product(got, exact(a), exact(b), torch.bfloat16)
    assert torch.equal(got, nv.matmul_fp8(a, b))
    assert nv.device_status() == 0


@pytest.mark.parametrize("block_rows", [1, 128])
def test_clusters_that_join_tile_after_tile(block_rows):
    """23 members of 65 rows are 46 tiles of 64 rows, more than there are clusters of eight CTAs at a time."""
    counts = [65] * 23 + [5]
    offsets, off = member_offsets(counts)
    a, b = operand(off[-1], 2064, 1, 1), operand(120, 2064, block_rows, 2, lead=(len(counts),))
    got = nv.matmul_fp8_grouped(a, b, offsets, out_dtype=torch.float32)
    av, bv = exact(a), exact(b)
    for e in range(len(counts)):
        check_product(got[off[e]:off[e + 1]], av[off[e]:off[e + 1]], bv[e], torch.float32)
    assert torch.equal(got, nv.matmul_fp8_grouped(a, b, offsets, out_dtype=torch.float32))
    assert nv.device_status() == 0


def test_scales_that_start_off_a_boundary():
    """Members that start at any row, and widths that are no multiples of four: scales with a row each, 4-byte aligned."""
    counts = [301, 258, 0, 515, 130]
    offsets, off = member_offsets(counts)
    for N, pad in ((260, 0), (259, 0), (260, 1)):
        a, b = operand(off[-1] + 4, 528, 1, 1), operand(N, 528, 1, 2, lead=(len(counts),))
        if pad:  # the same scales, one float further into their storage
            storage = torch.cat([torch.zeros(1, device="cuda"), b.scale.flatten()])
            b = nv.FP8Operand(b.data, storage[1:].view(b.scale.shape), 1)
        got = nv.matmul_fp8_grouped(a, b, offsets, out_dtype=torch.float32)
        av, bv = exact(a), exact(b)
        for e in range(len(counts)):
            check_product(got[off[e]:off[e + 1]], av[off[e]:off[e + 1]], bv[e], torch.float32)
        assert nv.device_status() == 0
    a, b = operand(2503, 400, 1, 3), operand(2301, 400, 1, 4)
    check_product(nv.matmul_fp8(a, b, out_dtype=torch.float32), exact(a), exact(b), torch.float32)
    assert nv.device_status() == 0
