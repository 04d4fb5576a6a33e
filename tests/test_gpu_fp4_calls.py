"""How the 4-bit operators may be called: views, streams, graphs, two at once; what they refuse; extremes of their inputs."""
import threading

import pytest
import torch

import nvfp4_block_scaled_amax_gb300 as nv
from fp4_testutil import operand, random_parts, values

pytestmark = pytest.mark.gpu

U32, U16 = 2.0 ** -24, 2.0 ** -8


def experts(E, H, F, block, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = lambda *s: torch.randn(*s, generator=g, device="cuda") * 0.1  # noqa: E731
    return nv.quantize_experts(w(E, 2 * F, H), block), nv.quantize_experts(w(E, H, F), block)


def layer_inputs(T, topk, E, H, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(T, H, generator=g, device="cuda").bfloat16(),
            torch.randint(0, E, (T, topk), generator=g, device="cuda", dtype=torch.int32),
            torch.rand(T, topk, generator=g, device="cuda"))


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("m,n,k", [(5, 300, 1056), (200, 300, 1056), (40, 260, 4128), (200, 300, 1024),
                                   (150, 400, 1280)])
def test_scales_at_any_address(m, n, k, block):
    pa, pb = random_parts(m, k, block, 1, True), random_parts(n, k, block, 2, True)
    want = nv.matmul_fp4(operand(pa, block), operand(pb, block))
    for shift in (1, 2, 3, 5, 7, 8, 11, 15, 16):
        ops = []
        for data, scale, amax in (pa, pb):
            room = torch.full((scale.numel() + 64,), 255, dtype=torch.uint8, device="cuda")  # NaN on both sides
            room[shift:shift + scale.numel()] = scale.cuda().reshape(-1)
            more = None
            if amax is not None:
                more = torch.full((4,), float("nan"), device="cuda")
                more[3] = amax[0]
                more = more[3:]
            ops.append(nv.FP4Operand(data.cuda(), room[shift:shift + scale.numel()], more, block))
        assert torch.equal(nv.matmul_fp4(*ops), want)


def test_out_and_side_stream():
    a, b = operand(random_parts(70, 256, 16, 1, True), 16), operand(random_parts(96, 256, 16, 2, True), 16)
    want = nv.matmul_fp4(a, b)
    out = torch.full((70, 96), float("nan"), device="cuda", dtype=torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert nv.matmul_fp4(a, b, out=out) is out
    side.synchronize()
    assert torch.equal(out, want)
    full = torch.full((100, 96), 7.0, device="cuda", dtype=torch.bfloat16)
    nv.matmul_fp4(a, b, out=full[15:85])
    assert torch.equal(full[15:85], want) and bool((full[:15] == 7).all()) and bool((full[85:] == 7).all())
    full = torch.full((80, 91), 7.0, device="cuda")  # rows off 16-byte boundaries, and rows behind the last
    c = operand(random_parts(91, 256, 16, 3, True), 16)
    nv.matmul_fp4(a, c, out=full[:70])
    assert torch.equal(full[:70], nv.matmul_fp4(a, c, out_dtype=torch.float32)) and bool((full[70:] == 7).all())


@pytest.mark.parametrize("T,topk", [(1, 2), (2, 4), (6, 2), (20, 3)])
def test_layer_in_graphs(T, topk):
    """Captured twice, replayed on two streams at once, with other inputs in place; beside eager calls."""
    E, H, F = 6, 512, 256
    up, down = experts(E, H, F, 16, 1)
    x, ids, gates = layer_inputs(T, topk, E, H, 2)
    nv.expert_mlp(x, up, down, ids, gates)
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        with torch.cuda.stream(s):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                outs.append(nv.expert_mlp(x, up, down, ids, gates))
        graphs.append(g)
    for seed in (3, 4, 5):
        for dst, src in zip((x, ids, gates), layer_inputs(T, topk, E, H, seed)):
            dst.copy_(src)
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                for _ in range(5):
                    g.replay()
        eager = nv.expert_mlp(x, up, down, ids, gates)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], eager) and torch.equal(outs[1], eager)
    assert nv.device_status() == 0


def test_product_and_cast_in_a_graph():
    x = torch.randn(160, 256, device="cuda").bfloat16()
    w = nv.quantize_mxfp4(torch.randn(192, 256, device="cuda")).row
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        nv.matmul_fp4(nv.quantize_mxfp4(x).row, w)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            y = nv.matmul_fp4(nv.quantize_mxfp4(x).row, w)
        for seed in range(3):
            x.copy_(torch.randn(160, 256, device="cuda") * (seed + 1))
            g.replay()
            s.synchronize()
            assert torch.equal(y, nv.matmul_fp4(nv.quantize_mxfp4(x).row, w))


def test_two_threads():
    """Calls of two threads, each on its own stream and both on one."""
    E, H, F = 4, 384, 320
    up, down = experts(E, H, F, 32, 1)
    inputs = [layer_inputs(3 + 9 * i, 2, E, H, 10 + i) for i in range(2)]
    want = [nv.expert_mlp(x, up, down, ids, gates) for x, ids, gates in inputs]
    torch.cuda.synchronize()
    for streams in ([torch.cuda.Stream(), torch.cuda.Stream()], [torch.cuda.Stream()] * 2):
        wrong = []

        def work(i):
            x, ids, gates = inputs[i]
            with torch.cuda.stream(streams[i]):
                for _ in range(30):
                    if not torch.equal(nv.expert_mlp(x, up, down, ids, gates), want[i]):
                        wrong.append(i)
        threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert not wrong


@pytest.mark.parametrize("m,n", [(6, 200), (150, 300)])
def test_factors_far_apart(m, n):
    """amax / 2688 of either side from subnormal to the largest numbers: no step leaves FP32 unless the result does."""
    k = 128
    (da, sa, _), (db, sb, _) = random_parts(m, k, 16, 1, True), random_parts(n, k, 16, 2, True)
    for fa, fb in ((1e-30, 1e30), (3e38, 1e-37), (1e-37, 3e38), (1e-22, 1e-20), (1e20, 1e18), (1e-40, 1e30), (0.0, 1.0)):
        aa, ab = torch.tensor([fa]), torch.tensor([fb])
        y = nv.matmul_fp4(operand((da, sa, aa), 16), operand((db, sb, ab), 16), out_dtype=torch.float32).cpu().double()
        # the factors are FP32 quotients, off by half a unit (of the smallest number, where they are subnormal)
        f = (aa / 2688.0).double(), (ab / 2688.0).double()
        want = (values(da, sa, None, 16) @ values(db, sb, None, 16).t()) * (f[0] * f[1])
        big = want.abs() > 3.4e38
        assert bool(((y - want).abs() <= 4 * U32 * want.abs() + 2.0 ** -148)[~big].all())
        assert bool(torch.isinf(y[big]).all())


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,n,per_a,per_b", [(6, 200, True, True), (40, 130, True, False), (40, 130, False, True),
                                             (150, 300, True, True), (300, 520, False, True), (260, 256, True, False)])
def test_factors_of_rows_far_apart(m, n, per_a, per_b, out_dtype):
    """An amax for each row of either side or both, of every size side by side, zero and not finite."""
    k = 128
    (da, sa, _), (db, sb, _) = random_parts(m, k, 16, 1, True), random_parts(n, k, 16, 2, True)
    da[3], db[5] = 0, 0                                 # sums of zero under each of them
    sizes = torch.tensor([1.0, 1e-30, 3e38, 2688.0, 1e-37, 1e-22, 7e4, 1e20, 1e-40, 1e18, 0.0, float("inf"), float("nan")])
    g = torch.Generator().manual_seed(m)
    for plain in (True, False):                         # columns that one product serves, and columns of all sorts
        def amaxes(rows, per):
            pick = torch.randint(0, 4 if plain else len(sizes), (rows if per else 1,), generator=g)
            some = torch.tensor([0, 3, 6, 0]) if plain else torch.arange(len(sizes))
            return sizes[some[pick]] if per else torch.tensor([1e-3])
        aa, ab = amaxes(m, per_a), amaxes(n, per_b)
        y = nv.matmul_fp4(operand((da, sa, aa), 16), operand((db, sb, ab), 16), out_dtype=out_dtype).cpu().double()
        f = (aa / 2688.0).double()[:, None] * (ab / 2688.0).double()
        want = (values(da, sa, None, 16) @ values(db, sb, None, 16).t()) * f
        # sums exact; the factors' product or two steps, and the rounding to FP32's or BF16's numbers
        u, least, most = (U16, 2.0 ** -133, 3.3895e38) if out_dtype == torch.bfloat16 else (U32, 2.0 ** -148, 3.4e38)
        nan, big = want.isnan(), want.abs() > most
        assert bool(y[nan].isnan().all()) and bool((y[big] * want[big].sign() >= most * (1 - 2 * u)).all())
        fine = ~(nan | big)
        assert bool(((y - want).abs() <= (4 * U32 + u) * want.abs() + least)[fine].all())


def test_nan_scale_stays_in_its_row():
    for block in (16, 32):
        for m, n in ((4, 130), (130, 260)):
            pa, pb = random_parts(m, 256, block, 1, True), random_parts(n, 256, block, 2, True)
            want = nv.matmul_fp4(operand(pa, block), operand(pb, block))
            pa[1][2, 3] = 255 if block == 32 else 127
            pb[1][77, 1] = 255 if block == 32 else 127
            y = nv.matmul_fp4(operand(pa, block), operand(pb, block))
            hit = torch.zeros(m, n, dtype=torch.bool, device="cuda")
            hit[2], hit[:, 77] = True, True
            assert bool(torch.isnan(y[hit]).all()) and torch.equal(y[~hit], want[~hit])


def test_amax_per_row():
    """The row-scaled cast's operand, on either side."""
    g = torch.Generator().manual_seed(1)
    x = (torch.randn(9, 128, generator=g) * torch.logspace(-6, 6, 9)[:, None]).bfloat16().cuda()
    w = torch.randn(140, 128, generator=g).bfloat16().cuda()
    q, p = nv.quantize(x, "row_scaled"), nv.quantize(w, "row_scaled")
    a, b = nv.dequantize_fp4(q.row, torch.float32).double(), nv.dequantize_fp4(p.row, torch.float32).double()
    for s, t, u, v in ((q, p, a, b), (p, q, b, a)):
        y = nv.matmul_fp4(s.row, t.row, out_dtype=torch.float32)
        assert bool(((y.double() - u @ v.t()).abs() <= 140 * U32 * (u.abs() @ v.abs().t())).all())


def test_refusals():
    a, b = operand(random_parts(8, 64, 16, 1), 16), operand(random_parts(8, 64, 16, 2), 16)
    for bad, error in ((nv.FP4Operand(b.data[:, :16].contiguous(), b.scale, b.amax), ValueError),
                       (nv.FP4Operand(b.data.t(), b.scale, b.amax), ValueError),
                       (nv.FP4Operand(b.data, b.scale.reshape(-1)[:31], b.amax), ValueError),
                       (nv.FP4Operand(b.data, b.scale), TypeError),
                       (nv.FP4Operand(b.data, b.scale, b.amax.double()), TypeError),
                       (nv.FP4Operand(b.data, b.scale, torch.ones(3, device="cuda")), ValueError),
                       (nv.FP4Operand(b.data, b.scale, torch.ones(1)), ValueError),
                       (nv.FP4Operand(b.data, b.scale.cpu(), b.amax), ValueError),
                       (nv.FP4Operand(b.data, b.scale, b.amax, 8), ValueError),
                       (nv.FP4Operand(b.data, b.scale.reshape(-1)[:16].contiguous(), None, 32), ValueError),
                       (nv.FP4Operand(b.data, b.scale, b.amax, 16, swizzled=True), nv.NVFP4Error),
                       (nv.FP4Operand(b.data.view(torch.int8), b.scale, b.amax), TypeError)):
        with pytest.raises(error):
            nv.matmul_fp4(a, bad)
        with pytest.raises(error):
            nv.matmul_fp4(bad, a)
    with pytest.raises(TypeError):
        nv.matmul_fp4(a, b, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        nv.matmul_fp4(a, b, out=torch.empty(8, 9, device="cuda"))
    with pytest.raises(ValueError):
        nv.matmul_fp4(a, b, out=torch.empty(8, 16, device="cuda")[:, ::2])
    with pytest.raises(TypeError):
        nv.quantize_mxfp4(torch.zeros(32, 32, device="cuda").half())
    with pytest.raises(ValueError):
        nv.quantize_mxfp4(torch.zeros(32, 64, device="cuda")[:, ::2])
    with pytest.raises(nv.NVFP4Error):
        nv.quantize_mxfp4(torch.zeros(32, 64, device="cuda"), swizzled=True)
    with pytest.raises(nv.NVFP4Error):
        nv.quantize_mxfp4(torch.zeros(32, 64, device="cuda"), rowwise=False)


def test_layer_refusals():
    up, down = experts(3, 64, 32, 16, 1)
    x, ids, gates = layer_inputs(4, 2, 3, 64, 2)
    other = nv.quantize_experts(torch.zeros(3, 64, 32, device="cuda"), 32)
    for args, error in (((x.float(), up, down, ids, gates), TypeError), ((x, up, down, ids.long(), gates), TypeError),
                        ((x, up, down, ids, gates.half()), TypeError), ((x, down, up, ids, gates), ValueError),
                        ((x, up, other, ids, gates), ValueError), ((x[:3], up, down, ids, gates), ValueError),
                        ((x, up, down, ids, gates[:, :1]), ValueError), ((x[:, :32].contiguous(), up, down, ids, gates), ValueError),
                        ((x.cpu(), up, down, ids, gates), ValueError), ((x, up, down, ids.cpu(), gates), ValueError),
                        ((x, up, down, ids, gates.t().contiguous().t()), ValueError),
                        ((x.repeat(200, 1), up, down, ids.repeat(200, 1), gates.repeat(200, 1)), ValueError)):
        with pytest.raises(error):
            nv.expert_mlp(*args)
    swizzled = nv.FP4Operand(up.data, up.scale, up.amax, 16, swizzled=True)
    with pytest.raises(ValueError, match="compact"):
        nv.expert_mlp(x, swizzled, down, ids, gates)
    with pytest.raises(ValueError):
        nv.expert_mlp(x, up, down, ids, gates, out=torch.empty(4, 64, device="cuda"))
    empty = nv.expert_mlp(x[:0], up, down, ids[:0], gates[:0])
    assert empty.shape == (0, 64)
    out = torch.empty_like(x)
    assert nv.expert_mlp(x, up, down, ids, gates, out=out) is out
    assert torch.equal(out, nv.expert_mlp(x, up, down, ids, gates))
