"""The expert layer end to end: exact on inputs that the casts keep, close on ordinary ones."""
import pytest
import torch

import nvfp4_block_scaled_amax_gb300 as nv
from nvfp4_block_scaled_amax_gb300.experts import expert_layer, expert_layer_grad

pytestmark = pytest.mark.gpu


def reference(x, w, ids, gates, dy):
    """y and its gradients in 64 bits through autograd."""
    x, w, gates = (t.double().requires_grad_() for t in (x, w, gates))
    y = torch.zeros(x.shape[0], w.shape[1], dtype=torch.float64)
    for j in range(ids.shape[1]):
        there = (ids[:, j] >= 0) & (ids[:, j] < w.shape[0])
        part = torch.einsum("tnk,tk->tn", w[ids[there, j].long()], x[there])
        y = y.index_add(0, there.nonzero()[:, 0], gates[there, j, None] * part)
    y.backward(dy.double())
    return y.detach(), x.grad, w.grad, gates.grad


def inputs(T, topk, E, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, K, generator=g).bfloat16()
    w = (torch.randn(E, N, K, generator=g) * 0.05).bfloat16()
    ids = torch.randint(-1, E, (T, topk), generator=g, dtype=torch.int32)
    ids[0] = -1
    gates = torch.softmax(torch.randn(T, topk, generator=g), 1)
    return x, w, ids, gates, torch.randn(T, N, generator=g).bfloat16()


@pytest.mark.parametrize("T,topk,E,N,K", [(200, 2, 4, 144, 272), (37, 3, 9, 64, 128), (700, 2, 5, 256, 384)])
def test_layer_and_gradient(T, topk, E, N, K):
    x, w, ids, gates, dy = inputs(T, topk, E, N, K, seed=T)
    y, saved = expert_layer(x.cuda(), w.cuda(), ids.cuda(), gates.cuda())
    dx, dw, dg = expert_layer_grad(dy.cuda(), saved)
    # E4M3 keeps 4 significant bits: each factor is off by 2^-4 at most, about 2^-4 / sqrt(3) on average and independent
    # in every term, so a product of two casts is off by about 0.05 of its norm; 2^-4 is not reached
    for got, want in zip((y, dx, dw, dg), reference(x, w, ids, gates, dy)):
        assert float((got.cpu().double() - want).norm() / want.norm()) < 2.0 ** -4
    assert bool((y[0] == 0).all()) and bool((dx[0] == 0).all()) and bool((dg[0] == 0).all())
    served, nothing = expert_layer(x.cuda(), saved.weights, ids.cuda(), gates.cuda(), training=False)
    assert nothing is None
    # the same rows through the same products: padding changes where a row lies, not what is summed
    assert float((served.double() - y.double()).norm() / y.double().norm()) < 2.0 ** -8
    assert nv.device_status() == 0


def test_layer_is_exact_on_small_integers():
    """Gates 1, and inputs whose blocks have maximum 7 * 2^6 = 448: no cast rounds and every sum is an exact integer
    times 2^12, which bfloat16 rounds once at the end of the product."""
    T, E, N, K = 150, 3, 128, 256
    g = torch.Generator().manual_seed(3)
    x = torch.randint(-7, 8, (T, K), generator=g).float()
    w = torch.randint(-7, 8, (E, N, K), generator=g).float()
    x[:, ::32], w[:, ::32, ::32] = 7.0, 7.0
    ids = torch.randint(0, E, (T, 1), generator=g, dtype=torch.int32)
    y, _ = expert_layer((x * 64).bfloat16().cuda(), (w * 64).cuda(), ids.cuda(), torch.ones(T, 1).cuda(),
                        training=False)
    want = torch.einsum("tnk,tk->tn", w[ids[:, 0].long()].double(), x.double()) * 4096
    assert torch.equal(y.cpu(), want.bfloat16())
