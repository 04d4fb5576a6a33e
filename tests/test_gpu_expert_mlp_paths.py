"""The gated expert layer on either side of the rule between two launches and four or five: one or two tokens whose x does
not stay in shared memory beside so many tiles, and long inner sizes, which one cluster sums."""
import pytest
import torch

import nvfp4_block_scaled_amax_gb300 as nv
from test_gpu_expert_mlp_amax import layer_inputs, operand, selecting_layer, selecting_values

pytestmark = pytest.mark.gpu

U32, U16 = 2.0 ** -24, 2.0 ** -8


@pytest.mark.parametrize("T,topk,E,H,F", [(2, 4, 8, 3360, 1280), (1, 8, 8, 3360, 1280), (2, 4, 8, 3360, 96), (2, 4, 8, 320, 3360),
                                          (1, 2, 3, 10240, 160), (2, 4, 9, 160, 2336), (1, 1, 2, 10240, 4160)])
def test_hidden_values_one_by_one(T, topk, E, H, F):
    """As in test_gpu_expert_mlp_amax: exact sums up (6 * 2^8 * 3 for each of 10240 elements stay below 2^24 multiples of
    2^4), and one hidden value an output, held to 2^-21 of a scale that is 9 / 48 of its block's largest or 2^-19 of its row's."""
    up, down = selecting_layer(E, H, F, T + topk)
    x, ids, gates = layer_inputs(T, topk, E, H, 7)
    gates[:, 1:] = 0.0
    y = nv.expert_mlp(x.cuda(), operand(up), operand(down), ids.cuda(), gates.cuda()).cpu().double()
    at = torch.arange(H) % F
    for t in range(T):
        e = int(ids[t, 0])
        s = selecting_values([p[e] for p in up]) @ x[t].double()
        h = s[:F] / (1 + torch.exp(-s[:F])) * s[F:]
        block = h.abs().view(-1, 16).amax(1).repeat_interleave(16)
        off = 12 * U32 * h.abs() + 2.0 ** -21 * (1.125 / 6 * block + 2.0 ** -19 * h.abs().max()) * 1.01
        assert bool(((64 * y[t] - h[at]).abs() <= (off + U16 * (h.abs() + off))[at]).all())
    assert nv.device_status() == 0
