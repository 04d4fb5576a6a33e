"""The 4-bit linear layer end to end: against 64-bit products of what its casts stand for, and against differences."""
import pytest
import torch

import nvfp4_block_scaled_amax_gb300 as nv
from nvfp4_block_scaled_amax_gb300.linear import linear_layer, linear_layer_grad, quantize_linear

pytestmark = pytest.mark.gpu

U32, U16 = 2.0 ** -24, 2.0 ** -8


def check(got, a, b):
    """got: the product of the values of the operands a and b^T, summed in FP32 and rounded once."""
    a, b = nv.dequantize_fp4(a, torch.float32).double(), nv.dequantize_fp4(b, torch.float32).double()
    want = a @ b.t()
    tol = (a.shape[1] + 6) * U32 * (a.abs() @ b.abs().t()) + (U16 if got.dtype == torch.bfloat16 else 0.0) * want.abs()
    assert bool(((got.double() - want).abs() <= tol * 1.001).all())


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,N,K", [(32, 64, 96), (160, 96, 288), (256, 384, 640), (128, 128, 128), (480, 1056, 2080)])
def test_layer_and_gradient(T, N, K, dtype, fmt):
    g = torch.Generator().manual_seed(T + N)
    x, dy = torch.randn(T, K, generator=g).to(dtype).cuda(), torch.randn(T, N, generator=g).to(dtype).cuda()
    w = (torch.randn(N, K, generator=g) * 0.05).cuda()
    y, saved = linear_layer(x, w, format=fmt)
    assert y.shape == (T, N) and y.dtype == dtype
    check(y, saved.x.row, saved.weight.row)
    dx, dw = linear_layer_grad(dy, saved)
    assert dx.shape == (T, K) and dx.dtype == dtype and dw.shape == (N, K) and dw.dtype == torch.float32
    q = nv.quantize_mxfp4(dy, colwise=True) if fmt == "mxfp4" else nv.quantize(dy, "1d")
    check(dx, q.row, saved.weight.col)
    check(dw, q.col, saved.x.col)
    # four bits keep about three significant ones: products are off by some percent of their norm
    for got, want in ((y, x.double() @ w.double().t()), (dx, dy.double() @ w.double()), (dw, dy.double().t() @ x.double())):
        assert float((got.double() - want).norm() / want.norm()) < 0.25
    served, nothing = linear_layer(x, saved.weight, format=fmt, training=False)
    assert nothing is None and torch.equal(served, y)
    one, _ = linear_layer(x[:1], quantize_linear(w, fmt, training=False), format=fmt, training=False)
    assert one.shape == (1, N)
    assert nv.device_status() == 0


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_gradient_is_the_difference(fmt):
    """On values that the casts keep (E2M1 numbers, a 6 in every block of both directions) the sums are exact, so the change
    of sum(y * dy) with one element is the gradient times the change.  MXFP4: to the last bit.  NVFP4: the factor 6 / 2688
    = 1 / 448 is no FP32 number; it is rounded once for each operand, their product once, and the sum times it once, so
    each output is off by at most 4 U32 of itself."""
    near = 0.0 if fmt == "mxfp4" else 4.001 * U32
    T, N, K = 64, 96, 128
    g = torch.Generator().manual_seed(7)
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0])

    def matrix(rows, cols):
        v = grid[torch.randint(0, 7, (rows, cols), generator=g)] * torch.where(torch.rand(rows, cols, generator=g) < 0.5, 1.0, -1.0)
        r, c = torch.meshgrid(torch.arange(rows), torch.arange(cols), indexing="ij")
        return torch.where((r + c) % 16 == 0, 6.0, v)

    x, w, dy = matrix(T, K), matrix(N, K), matrix(T, N)
    y, saved = linear_layer(x.cuda(), w.cuda(), format=fmt)
    dx, dw = linear_layer_grad(dy.cuda(), saved)
    for got, want in ((y, x.double() @ w.double().t()), (dx, dy.double() @ w.double()), (dw, dy.double().t() @ x.double())):
        assert bool(((got.cpu().double() - want).abs() <= near * want.abs()).all())

    def loss(x, w):
        terms = linear_layer(x.cuda(), w.cuda(), format=fmt)[0].cpu().double() * dy.double()
        return float(terms.sum()), near * float(terms.abs().sum())
    base, base_off = loss(x, w)
    for i in range(12):
        t, n, k = (int(torch.randint(0, s, (1,), generator=g)) for s in (T, N, K))
        if (t + k) % 16 and (n + k) % 16:
            for one, other, at, grad in ((x, x.clone(), (t, k), dx), (w, w.clone(), (n, k), dw)):
                other[at] = 3.0 if one[at] != 3.0 else -1.0
                changed, off = loss(other, w) if one is x else loss(x, other)
                want = float(grad[at].cpu().double() * (other[at] - one[at]))
                assert abs(changed - base - want) <= base_off + off + near * abs(want)


def test_refusals():
    x, w = torch.zeros(32, 64, device="cuda"), torch.zeros(32, 64, device="cuda")
    with pytest.raises(ValueError):
        linear_layer(x, w, format="fp4")
    with pytest.raises(ValueError):
        linear_layer(x[0], w)
    with pytest.raises(ValueError, match="column-wise"):
        linear_layer(x, quantize_linear(w, training=False))
    with pytest.raises(ValueError):
        linear_layer(x[:, :40].contiguous(), w[:, :40].contiguous())
    with pytest.raises(ValueError):
        linear_layer(x[:, :32].contiguous(), w)
