"""Tokens sorted by expert and joined again, against plain loops and 64-bit sums."""
import pytest
import torch

import nvfp4_block_scaled_amax_gb300 as nv

pytestmark = pytest.mark.gpu

U32, U16 = 2.0 ** -24, 2.0 ** -8  # half a unit in the last place, relative: FP32, BF16


def make_ids(T, topk, E, seed, drop=0.1):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, E, (T, topk), generator=g, dtype=torch.int32)
    if E > 2:
        ids[ids == E // 2] = 0  # an expert without rows
    lost = torch.rand(T, topk, generator=g) < drop
    ids[lost] = -1
    if T > 3:
        ids[2] = -1  # a token with nothing left
        ids[3, 0] = E  # one past the last expert: dropped as well
    return ids


def plan_by_loop(ids, E, align):
    flat = ids.reshape(-1).tolist()
    lists = [[s for s, e in enumerate(flat) if e == k] for k in range(E)]
    offsets, slots = [0], []
    for m in lists:
        slots += m + [-1] * (-len(m) % align)
        offsets.append(len(slots))
    cap = (len(flat) + E * (align - 1)) // align * align
    slots += [-1] * (cap - len(slots))
    rows = [-1] * len(flat)
    for r, s in enumerate(slots):
        if s >= 0:
            rows[s] = r
    return offsets, rows, slots


PLANS = [(1, 1, 1, 1), (1, 8, 128, 1), (5, 2, 8, 1), (33, 3, 7, 16), (257, 4, 32, 128), (1024, 2, 8, 1),
         (1025, 2, 8, 128), (700, 6, 1024, 1), (4099, 5, 33, 128), (40000, 8, 64, 16), (0, 2, 4, 128)]


@pytest.mark.parametrize("T,topk,E,align", PLANS)
def test_sort(T, topk, E, align):
    ids = make_ids(T, topk, E, seed=T + E)
    plan = nv.sort_tokens(ids.cuda(), E, align=align)
    offsets, rows, slots = plan_by_loop(ids, E, align)
    assert plan.offsets.tolist() == offsets
    assert plan.row_of_slot.reshape(-1).tolist() == rows
    assert plan.slot_of_row.tolist() == slots


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,topk,E,align,H", [(1, 1, 1, 1, 8), (5, 2, 8, 1, 1024), (33, 3, 7, 16, 72),
                                              (1025, 2, 8, 128, 520), (2100, 4, 16, 1, 2056), (3, 2, 4, 1, 20000),
                                              (64, 2, 8, 128, 5128)])
def test_dispatch_copies_rows(T, topk, E, align, H, dtype):
    ids = make_ids(T, topk, E, seed=H)
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(1)).to(dtype)
    x[0, :2] = torch.tensor([float("nan"), float("inf")])  # copied like anything else
    rows, plan = nv.dispatch_tokens(x.cuda(), ids.cuda(), E, align=align)
    offsets, _, slots = plan_by_loop(ids, E, align)
    want = torch.zeros(len(slots), H, dtype=dtype)
    for r, s in enumerate(slots):
        if s >= 0:
            want[r] = x[s // topk]
    kind = torch.int16 if dtype == torch.bfloat16 else torch.int32
    assert torch.equal(rows.cpu().view(kind), want.view(kind))
    assert plan.offsets.tolist() == offsets
    again = nv.gather_tokens(x.cuda(), plan)
    assert torch.equal(again.view(kind), rows.view(kind))


def combine_inputs(T, topk, E, align, H, dtype, seed):
    ids = make_ids(T, topk, E, seed=seed)
    plan = nv.sort_tokens(ids.cuda(), E, align=align)
    g = torch.Generator().manual_seed(seed)
    rows = torch.randn(plan.rows, H, generator=g).to(dtype)
    w = torch.rand(T, topk, generator=g)
    return plan, rows, w


CASES = [(1, 1, 1, 1, 8), (5, 2, 8, 1, 1024), (101, 2, 16, 1, 5120), (33, 3, 7, 16, 72), (513, 8, 32, 128, 520),
         (64, 1, 2, 128, 4104), (7, 64, 90, 1, 264), (3, 2, 4, 1, 20000)]


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,topk,E,align,H", CASES)
def test_combine(T, topk, E, align, H, dtype, weighted):
    plan, rows, w = combine_inputs(T, topk, E, align, H, dtype, seed=T + H)
    at = plan.row_of_slot.cpu().long()
    slots = plan.slot_of_row.cpu()
    rows[slots < 0] = float("nan")  # padding rows are never read
    y = nv.combine_tokens(rows.cuda(), plan, w.cuda() if weighted else None).cpu().double()
    part = torch.where((at >= 0)[..., None], rows[at.clamp(min=0)].double(), 0.0)
    part = part * (w.double()[..., None] if weighted else 1.0)
    want = part.sum(1)
    out = U16 if dtype == torch.bfloat16 else U32
    bound = (topk + 1) * U32 * part.abs().sum(1) * (1 + out) + out * want.abs()
    assert bool(((y - want).abs() <= bound).all())
    assert bool((y[(at < 0).all(1)] == 0).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,topk,E,align,H", CASES)
def test_combine_grad(T, topk, E, align, H, dtype):
    plan, rows, w = combine_inputs(T, topk, E, align, H, dtype, seed=T + H)
    at, slots = plan.row_of_slot.cpu().long(), plan.slot_of_row.cpu().long()
    rows[slots < 0] = float("nan")
    dy = torch.randn(T, H, generator=torch.Generator().manual_seed(9)).to(dtype)
    drows, dw = nv.combine_tokens_grad(dy.cuda(), rows.cuda(), plan, w.cuda())
    there = slots >= 0
    want = torch.zeros(plan.rows, H, dtype=torch.float64)
    want[there] = w.reshape(-1).double()[slots[there], None] * dy.double()[slots[there] // topk]
    out = U16 if dtype == torch.bfloat16 else 0.0
    assert bool(((drows.cpu().double() - want).abs() <= (out + 2 * U32) * want.abs()).all())
    part = torch.where((at >= 0)[..., None], rows[at.clamp(min=0)].double(), 0.0) * dy.double()[:, None]
    # a thread adds at most ceil(H / 128) + 8 terms in a row, the tree another 12 levels
    bound = (H / 128 + 24) * U32 * part.abs().sum(-1)
    assert bool(((dw.cpu().double() - part.sum(-1)).abs() <= bound).all())
    ones = nv.combine_tokens_grad(dy.cuda(), rows.cuda(), plan)[0]
    assert torch.equal(ones, nv.gather_tokens(dy.cuda(), plan))


def test_combine_gradient_against_differences():
    """<dy, y> is linear in the rows and in the weights: central differences are exact but for rounding."""
    T, topk, E, H = 19, 3, 5, 64
    plan, rows, w = combine_inputs(T, topk, E, 1, H, torch.float32, seed=4)
    g = torch.Generator().manual_seed(5)
    dy = torch.randn(T, H, generator=g)
    drows, dw = (t.cpu().double() for t in nv.combine_tokens_grad(dy.cuda(), rows.cuda(), plan, w.cuda()))

    def loss(r, v):
        return float((nv.combine_tokens(r.cuda(), plan, v.cuda()).cpu().double() * dy.double()).sum())
    for seed in range(4):
        g.manual_seed(seed)
        dr, dv = torch.randn(rows.shape, generator=g), torch.randn(w.shape, generator=g)
        size = float(rows.abs().sum())
        for at, got in (((dr, 0 * dv), (drows * dr.double()).sum()), ((0 * dr, dv), (dw * dv.double()).sum())):
            diff = (loss(rows + at[0], w + at[1]) - loss(rows - at[0], w - at[1])) / 2
            # inputs, products and sums each round; no sum of magnitudes here exceeds 100 * size
            assert abs(diff - float(got)) <= 16 * U32 * 100 * size
    # gather and its gradient are adjoint
    x = torch.randn(T, H, generator=g)
    r = torch.randn(plan.rows, H, generator=g)
    left = (nv.gather_tokens(x.cuda(), plan).cpu().double() * r.double()).sum()
    right = (x.double() * nv.gather_tokens_grad(r.cuda(), plan).cpu().double()).sum()
    assert abs(float(left - right)) <= 8 * U32 * float((x.abs().sum() * r.abs().max()))


def test_dispatch_then_combine_on_another_stream():
    T, topk, E, H = 300, 2, 8, 256
    ids = make_ids(T, topk, E, seed=1)
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(2))
    xd, idd = x.cuda(), ids.cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        rows, plan = nv.dispatch_tokens(xd, idd, E, align=16)
        y = nv.combine_tokens(rows, plan)
    s.synchronize()
    kept = (plan.row_of_slot.cpu() >= 0).sum(1)
    assert torch.equal(y.cpu(), x * kept[:, None])


def test_dispatch_in_a_graph():
    T, topk, E, H = 1500, 2, 8, 64
    ids, x = make_ids(T, topk, E, seed=1).cuda(), torch.randn(T, H, device="cuda")
    nv.dispatch_tokens(x, ids, E)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rows, plan = nv.dispatch_tokens(x, ids, E)
        y = nv.combine_tokens(rows, plan)
    for seed in (2, 3):
        ids.copy_(make_ids(T, topk, E, seed=seed))
        x.normal_()
        g.replay()
        torch.cuda.synchronize()
        kept = (plan.row_of_slot >= 0).sum(1)
        assert plan.offsets.tolist() == plan_by_loop(ids.cpu(), E, 1)[0]
        assert torch.allclose(y, x * kept[:, None], rtol=2 * U32, atol=0)


def test_refusals():
    x = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    ids = torch.zeros(4, 2, device="cuda", dtype=torch.int32)
    rows, plan = nv.dispatch_tokens(x, ids, 2)
    w = torch.ones(4, 2, device="cuda")
    for err, call in [
            (TypeError, lambda: nv.dispatch_tokens(x.half(), ids, 2)),
            (TypeError, lambda: nv.dispatch_tokens(x, ids.long(), 2)),
            (ValueError, lambda: nv.dispatch_tokens(x, ids[:3], 2)),
            (ValueError, lambda: nv.dispatch_tokens(x.t(), ids, 2)),
            (ValueError, lambda: nv.dispatch_tokens(x.cpu(), ids, 2)),
            (ValueError, lambda: nv.dispatch_tokens(x, ids, 0)),
            (ValueError, lambda: nv.dispatch_tokens(x, ids, 1025)),
            (ValueError, lambda: nv.dispatch_tokens(x, ids, 2, align=0)),
            (nv.NVFP4Error, lambda: nv.dispatch_tokens(x[:, :4].contiguous(), ids, 2)),
            (ValueError, lambda: nv.gather_tokens(x[:3], plan)),
            (ValueError, lambda: nv.combine_tokens(rows[:-1], plan, w)),
            (ValueError, lambda: nv.combine_tokens(rows, plan, w[:, :1])),
            (ValueError, lambda: nv.combine_tokens(rows, plan, w.double())),
            (ValueError, lambda: nv.combine_tokens_grad(x[:, :32].contiguous(), rows, plan, w)),
            (TypeError, lambda: nv.combine_tokens_grad(x.float(), rows, plan, w))]:
        with pytest.raises(err):
            call()


@pytest.mark.parametrize("T,topk,E,align", [(1024, 2, 32, 128), (1024, 2, 33, 128), (683, 3, 32, 100), (512, 4, 700, 1),
                                            (2048, 1, 1, 600), (300, 2, 3, 1000), (2049, 1, 40, 16)])
def test_dispatch_at_the_limits_of_one_launch(T, topk, E, align):
    """2048 slots, 6144 rows; members padded by more rows than a CTA has threads; more experts than threads."""
    ids = make_ids(T, topk, E, seed=T + align)
    x = torch.randn(T, 72, generator=torch.Generator().manual_seed(1)).bfloat16()
    rows, plan = nv.dispatch_tokens(x.cuda(), ids.cuda(), E, align=align)
    offsets, row_of_slot, slots = plan_by_loop(ids, E, align)
    s = torch.tensor(slots)
    want = torch.where((s >= 0)[:, None], x[s.clamp(min=0) // topk], torch.zeros((), dtype=torch.bfloat16))
    assert torch.equal(rows.cpu(), want)
    assert plan.offsets.tolist() == offsets and plan.slot_of_row.tolist() == slots
    assert plan.row_of_slot.flatten().tolist() == row_of_slot
