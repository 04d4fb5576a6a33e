"""4-bit operands that are written again, in place, right before a call: weights that are reloaded or swapped, and casts
into memory that earlier calls read."""
import pytest
import torch

import nvfp4_block_scaled_amax_gb300 as nv
from fp4_testutil import operand, random_parts
from test_gpu_expert_mlp import stack

pytestmark = pytest.mark.gpu

CALLS = 60


def parts_of(q):
    return [t for t in (q.data, q.scale, q.amax) if t is not None]


def copy_into(to, q):
    for a, b in zip(parts_of(to), parts_of(q)):
        a.copy_(b)


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("T,topk", [(1, 2), (2, 4), (12, 2), (40, 3)])
def test_experts_written_just_before(T, topk, block):
    """Codes, scales and amaxes of both stacks in the same memory, other ones for every call."""
    E, H, F, n = 5, 320, 160, 4
    g = torch.Generator().manual_seed(T)
    sets = [(stack(E, 2 * F, H, block, 10 * i, H ** -0.5)[0], stack(E, H, F, block, 10 * i + 5, F ** -0.5)[0]) for i in range(n)]
    x = torch.randn(T, H, generator=g).bfloat16().cuda()
    ids = torch.randint(0, E, (T, topk), generator=g, dtype=torch.int32).cuda()
    gates = torch.rand(T, topk, generator=g).cuda()
    want = []
    for up, down in sets:
        want.append(nv.expert_mlp(x, up, down, ids, gates))
        torch.cuda.synchronize()
    assert not torch.equal(want[0], want[1])
    up, down = (nv.FP4Operand(*(None if t is None else t.clone() for t in (q.data, q.scale, q.amax)), block) for q in sets[0])
    out = torch.empty(CALLS, T, H, dtype=torch.bfloat16, device="cuda")
    order = torch.randint(0, n, (CALLS,), generator=g).tolist()
    for k, i in enumerate(order):
        copy_into(up, sets[i][0])
        copy_into(down, sets[i][1])
        nv.expert_mlp(x, up, down, ids, gates, out=out[k])
    for k, i in enumerate(order):
        assert torch.equal(out[k], want[i])
    assert nv.device_status() == 0


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("m,n,k", [(3, 300, 1056), (3, 256, 1024), (200, 300, 1056), (200, 256, 1024)])
def test_products_of_operands_written_just_before(m, n, k, block):
    g = torch.Generator().manual_seed(m)
    sets = [(operand(random_parts(m, k, block, 2 * i, True), block), operand(random_parts(n, k, block, 2 * i + 1, True), block))
            for i in range(4)]
    want = [nv.matmul_fp4(a, b) for a, b in sets]
    read = [nv.dequantize_fp4(b) for _, b in sets]
    a, b = (nv.FP4Operand(*(None if t is None else t.clone() for t in (q.data, q.scale, q.amax)), block) for q in sets[0])
    out, back = [], []
    order = torch.randint(0, 4, (CALLS,), generator=g).tolist()
    for c, i in enumerate(order):
        copy_into(a, sets[i][0])
        copy_into(b, sets[i][1])
        out.append(nv.matmul_fp4(a, b))
        back.append(nv.dequantize_fp4(b))
    for c, i in enumerate(order):
        assert torch.equal(out[c], want[i]) and torch.equal(back[c], read[i])


@pytest.mark.parametrize("M,N", [(1, 64), (32, 4096), (160, 1056)])
def test_casts_into_memory_just_read(M, N):
    """Cast, read back and multiply one matrix after the other, with nothing between the launches but their kernels."""
    xs = [torch.randn(M, N, generator=torch.Generator().manual_seed(i)).bfloat16().cuda() for i in range(4)]
    w = nv.quantize_mxfp4(torch.randn(96, N, generator=torch.Generator().manual_seed(9)).cuda()).row
    want = []
    for x in xs:
        q = nv.quantize_mxfp4(x).row
        want.append((nv.dequantize_fp4(q), nv.matmul_fp4(q, w)))
        torch.cuda.synchronize()
    del q
    got = []
    for c in range(CALLS):
        q = nv.quantize_mxfp4(xs[c % 4]).row
        got.append((nv.dequantize_fp4(q), nv.matmul_fp4(q, w)))
        del q                                        # its memory is the next cast's
    for c in range(CALLS):
        assert torch.equal(got[c][0], want[c % 4][0]) and torch.equal(got[c][1], want[c % 4][1])
