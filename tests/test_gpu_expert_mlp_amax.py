"""The gated expert layer over NVFP4 weights whose amax says little about the weights in use: what the hidden values are
held in goes by the values themselves."""
import pytest
import torch

import nvfp4_block_scaled_amax_gb300 as nv
from fp4_testutil import pack, scale_values, unpack

pytestmark = pytest.mark.gpu

U32, U16 = 2.0 ** -24, 2.0 ** -8
# (tokens, choices, experts): two launches for the first four, then segments of two, eight and sixteen tokens
COUNTS = [(1, 1, 1), (1, 8, 9), (2, 2, 4), (2, 4, 3), (1, 9, 12), (5, 2, 4), (40, 3, 4)]


def power_scales(shape, lo, hi, g):
    """E4M3 bytes of powers of two 2^lo .. 2^hi."""
    return (8 * (torch.randint(lo, hi + 1, shape, generator=g) + 7)).to(torch.uint8)


def shifted(scale, by):
    """The bytes of scales 2^-by times as large, powers of two all of them (down to 2^-9, which E4M3 holds)."""
    v = scale.view(torch.float8_e4m3fn).double() * 2.0 ** -by
    out = v.to(torch.float8_e4m3fn)
    assert bool((out.double() == v).all())
    return out.view(torch.uint8)


def selecting_layer(E, H, F, seed):
    """Parts of experts whose sums are exact, and whose second product picks hidden values one by one: the scales of the gate
    and up rows are powers of two, row o of the down matrix holds a single 1, at column o % F, with a scale of 2^8.  Their
    amaxes are 2688 2^-14, a factor of 2^-14."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 16, (E, 2 * F, H), generator=g).to(torch.uint8)
    up = pack(codes), power_scales((E, 2 * F, H // 16), 5, 8, g)
    down_codes = torch.zeros(E, H, F, dtype=torch.uint8)
    o = torch.arange(H)
    down_codes[:, o, o % F] = 2                      # 1.0
    scale = torch.full((E, H, F // 16), 8 * (8 + 7), dtype=torch.uint8)
    return up, (pack(down_codes), scale)


def operand(parts, by=0, amax=None):
    """The stack with scales 2^-by times as large and a factor 2^by times as large."""
    E = parts[0].shape[0]
    amax = torch.full((E,), 2688.0 * 2.0 ** (by - 14)) if amax is None else amax
    return nv.FP4Operand(parts[0].cuda(), shifted(parts[1], by).cuda(), amax.cuda(), 16)


def selecting_values(parts):
    return unpack(parts[0]) * scale_values(parts[1], 16).repeat_interleave(16, -1) * 2.0 ** -14


def layer_inputs(T, topk, E, H, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(-3, 4, (T, H), generator=g).float()
    x[:, ::16] = 3.0                                 # in every block: a scale of 1/2, codes 0, 2, 4 and 6
    ids = torch.stack([torch.randperm(E, generator=g)[:topk] if topk <= E else torch.randint(0, E, (topk,), generator=g)
                       for _ in range(T)]).int()
    return x.bfloat16(), ids, torch.ones(T, topk)


@pytest.mark.parametrize("T,topk,E", COUNTS)
def test_the_same_weights_with_another_amax(T, topk, E):
    """A factor that is a power of two larger and block scales that are smaller by it: the same numbers, so the same bits,
    up to a factor of 1 where the scales carry everything."""
    H, F = 288, 160
    up, down = selecting_layer(E, H, F, T + topk)
    x, ids, gates = (v.cuda() for v in layer_inputs(T, topk, E, H, 3))
    want = nv.expert_mlp(x, operand(up), operand(down), ids, gates)
    assert bool((want != 0).any())
    for by in (4, 6, 10, 14):
        assert torch.equal(nv.expert_mlp(x, operand(up, by), operand(down), ids, gates), want)
        assert torch.equal(nv.expert_mlp(x, operand(up, by), operand(down, by), ids, gates), want)
    assert nv.device_status() == 0


@pytest.mark.parametrize("T,topk,E", COUNTS)
@pytest.mark.parametrize("by", [0, 6, 14])
def test_hidden_values_one_by_one(T, topk, E, by):
    """Every output is one hidden value of the first choice (the others have gates of zero).

    The sums g and u are exact: x is held exactly by its first term, and code times scale times x is a multiple of 2^4 up to
    6 * 2^8 * 3, so 288 of them are whole multiples below 2^24.  SiLU and the product cost a handful of roundings in 32 bits.
    A block of 16 hidden values has a scale s of at most 9 / 8 of a sixth of its largest value (the next E4M3 number), or the
    smallest scale, 2^-9 of a unit that is at most 2^-10 of the row's largest value; its terms leave at most s 2^-15.  The
    picked value times 2^-6 is rounded to BF16 once."""
    H, F = 288, 160
    up, down = selecting_layer(E, H, F, T + topk + 1)
    x, ids, gates = layer_inputs(T, topk, E, H, 4)
    gates[:, 1:] = 0.0
    y = nv.expert_mlp(x.cuda(), operand(up, by), operand(down, by), ids.cuda(), gates.cuda()).cpu().double()
    v = selecting_values(up)
    for t in range(T):
        s = v[ids[t, 0].long()] @ x[t].double()
        h = s[:F] / (1 + torch.exp(-s[:F])) * s[F:]
        block = h.abs().view(-1, 16).amax(1).repeat_interleave(16)
        left = 2.0 ** -15 * (1.125 / 6 * block + 2.0 ** -19 * h.abs().max())
        off = 12 * U32 * h.abs() + left * 1.01
        at = torch.arange(H) % F
        assert bool(((64 * y[t] - h[at]).abs() <= (off + U16 * (h.abs() + off))[at]).all())


@pytest.mark.parametrize("T,topk,E", [(1, 2, 3), (2, 4, 3), (6, 2, 3), (40, 2, 3)])
@pytest.mark.parametrize("sigmas", [0, 50, 200, 1000, 4000])
def test_one_large_weight(T, topk, E, sigmas):
    """Normal weights with one of many standard deviations in every expert, cast as a user casts them."""
    H, F = 512, 384
    g = torch.Generator().manual_seed(sigmas)
    w_up, w_down = torch.randn(E, 2 * F, H, generator=g) * H ** -0.5, torch.randn(E, H, F, generator=g) * F ** -0.5
    if sigmas:
        w_up[:, 7, 11] = sigmas * H ** -0.5
    up, down = nv.quantize_experts(w_up.cuda()), nv.quantize_experts(w_down.cuda())
    x = torch.randn(T, H, generator=g).bfloat16().cuda()
    x[:, 11] = 0.0                                   # (the hidden values are those of the other weights)
    ids = torch.randint(0, E, (T, topk), generator=g, dtype=torch.int32).cuda()
    gates = torch.softmax(torch.randn(T, topk, generator=g), 1).cuda()
    y = nv.expert_mlp(x, up, down, ids, gates).double()
    check_norms(y, x, up, down, ids, gates)


def values_of(q):
    E, n, k2 = q.data.shape
    flat = nv.dequantize_fp4(nv.FP4Operand(q.data.view(E * n, k2), q.scale.view(E * n, -1),
                                           q.amax.expand(E).repeat_interleave(n).contiguous(), 16), torch.float32)
    return flat.view(E, n, 2 * k2).double()


def check_norms(y, x, up, down, ids, gates):
    """Rounding to BF16 is off by at most U16 of each output, so by at most U16 in the norm.  Sums of n products in 32 bits,
    in an order of the tensor cores' choice, are off by at most n U32 of their magnitudes' sum, which for n normal weights is
    0.64 sqrt(n) of the sums' deviation: 512 U32 14.5 = 4.4e-4 for g and u, so (1.1 + 0.6) 4.4e-4 / 0.6 = 1.2e-3 of the norm of
    h = silu(g) u, and 384 U32 12.5 = 2.9e-4 for y, together below 2^-9."""
    F = up.data.shape[1] // 2
    w_up, w_down = values_of(up), values_of(down)
    for t in range(x.shape[0]):
        want = torch.zeros_like(y[t])
        for e, gate in zip(ids[t].tolist(), gates[t].tolist()):
            s = w_up[e] @ x[t].double()
            want += gate * (w_down[e] @ (s[:F] * torch.sigmoid(s[:F]) * s[F:]))
        assert float((y[t] - want).norm()) <= (U16 + 2.0 ** -9) * float(want.norm())


@pytest.mark.parametrize("T,topk", [(1, 2), (2, 2), (6, 2), (40, 2)])
@pytest.mark.parametrize("larger", [1.0, 16.0, 64.0, 1000.0])
def test_one_amax_for_all_experts(T, topk, larger):
    """One amax for a stack with an expert that is much larger than the others, which the tokens do not choose."""
    E, H, F = 4, 512, 384
    g = torch.Generator().manual_seed(5)
    ops = []
    for n, k in ((2 * F, H), (H, F)):
        w = torch.randn(E, n, k, generator=g) * k ** -0.5
        w[3] *= larger
        q = nv.quantize(w.view(E * n, k).cuda(), "1d", colwise=False)
        ops.append(nv.FP4Operand(q.data_row.view(E, n, k // 2), q.scale_row.view(E, n, k // 16), q.amax_row, 16))
    x = torch.randn(T, H, generator=g).bfloat16().cuda()
    ids = torch.randint(0, 3, (T, topk), generator=g, dtype=torch.int32).cuda()
    gates = torch.softmax(torch.randn(T, topk, generator=g), 1).cuda()
    y = nv.expert_mlp(x, *ops, ids, gates).double()
    check_norms(y, x, *ops, ids, gates)
