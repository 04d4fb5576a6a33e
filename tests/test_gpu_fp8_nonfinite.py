"""Non-finite values through the cast in both types, both block shapes and both directions, and the expert layer in
FP32."""
import pytest
import torch

import nvfp4_block_scaled_amax_gb300 as nv
from nvfp4_block_scaled_amax_gb300.experts import expert_layer, expert_layer_grad

pytestmark = pytest.mark.gpu

BLOCK = 128
NAN, INF = float("nan"), float("inf")


def plain(x, block_rows):
    """(codes' values, scales) of one matrix on the CPU: maxima over the values that are no NaN, FP32 divisions."""
    M, N = x.shape
    m, n = -(-M // BLOCK) * BLOCK, -(-N // BLOCK) * BLOCK
    a = torch.nn.functional.pad(torch.where(torch.isnan(x), 0.0, x.abs()), (0, n - N, 0, m - M))
    a = a.view(m, -1, BLOCK).amax(-1) if block_rows == 1 else a.view(-1, BLOCK, n // BLOCK, BLOCK).amax((1, 3))
    a = a.clamp(min=2.0 ** -100)
    top = torch.full((), 448.0)
    scale, factor = a / top, top / a
    each = factor if block_rows == 1 else factor.repeat_interleave(BLOCK, 0)
    v = x * each[:M].repeat_interleave(BLOCK, 1)[:, :N]
    q = v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float()
    return torch.where(torch.isnan(v), NAN, q), scale[:M].t() if block_rows == 1 else scale


def same(a, b):
    return torch.equal(torch.nan_to_num(a, nan=12345.0), torch.nan_to_num(b, nan=12345.0))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("M,N", [(16, 16), (144, 272), (256, 384)])
def test_cast(M, N, block_rows, dtype):
    g = torch.Generator().manual_seed(M)
    x = torch.randn(M, N, generator=g).to(dtype).float()
    x[0, 0], x[1, 1] = NAN, -NAN             # beside finite values
    x[5, 3], x[M - 1, N - 1] = INF, -INF     # and in the last row and column
    x[7] = NAN                               # a whole row
    x[:, 9] = NAN                            # a whole column
    if M > 128:
        x[128:144, 128:256] = NAN            # (part of) a tile
        x[130, 258] = NAN
    q = nv.quantize_fp8(x.to(dtype).cuda(), block_rows=block_rows, colwise=True)
    for op, ref in ((q.row, x), (q.col, x.t().contiguous())):
        codes, scale = plain(ref, block_rows)
        assert same(op.scale.cpu(), scale)
        assert same(op.data.cpu().float(), codes)
        # nothing non-finite is lost: an infinity's block shows it, a NaN stays one
        back = op.dequantize().cpu()
        assert bool((~torch.isfinite(back))[~torch.isfinite(ref)].all())
    rows_only = nv.quantize_fp8(x.to(dtype).cuda(), block_rows=block_rows)
    assert torch.equal(rows_only.row.data.view(torch.uint8), q.row.data.view(torch.uint8))
    assert torch.equal(rows_only.row.scale, q.row.scale)


def test_expert_layer_in_fp32():
    """As in BF16, with inputs and outputs of 32 bits: E4M3 keeps four significant bits, so the norms' bound is the
    same; members of other sizes than the tiles, dropped choices among them."""
    T, topk, E, N, K = 300, 2, 5, 144, 272
    g = torch.Generator().manual_seed(7)
    x, dy = torch.randn(T, K, generator=g), torch.randn(T, N, generator=g)
    w = torch.randn(E, N, K, generator=g) * 0.05
    ids = torch.randint(-1, E, (T, topk), generator=g, dtype=torch.int32)
    gates = torch.softmax(torch.randn(T, topk, generator=g), 1)
    y, saved = expert_layer(x.cuda(), w.cuda(), ids.cuda(), gates.cuda())
    dx, dw, dg = expert_layer_grad(dy.cuda(), saved)
    assert y.dtype == dx.dtype == dw.dtype == dg.dtype == torch.float32
    xd, wd, gd = (t.double().requires_grad_() for t in (x, w, gates))
    want = torch.zeros(T, N, dtype=torch.float64)
    for j in range(topk):
        there = ids[:, j] >= 0
        part = torch.einsum("tnk,tk->tn", wd[ids[there, j].long()], xd[there])
        want = want.index_add(0, there.nonzero()[:, 0], gd[there, j, None] * part)
    want.backward(dy.double())
    for got, ref in ((y, want.detach()), (dx, xd.grad), (dw, wd.grad), (dg, gd.grad)):
        assert float((got.cpu().double() - ref).norm() / ref.norm()) < 2.0 ** -4
    served, _ = expert_layer(x.cuda(), saved.weights, ids.cuda(), gates.cuda(), training=False)
    # the same casts and products without padding: sums of 128 in another place differ by 2 (128 + 7) units of 2^-23 of the
    # sum of magnitudes at most, which is about sqrt(K) = 16 times the result: below 2^-10 of the norm
    assert float((served - y).double().norm() / y.double().norm()) < 2.0 ** -10
    assert nv.device_status() == 0
