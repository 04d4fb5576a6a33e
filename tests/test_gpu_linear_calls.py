"""The 4-bit linear layer captured into graphs."""
import pytest
import torch

import nvfp4_block_scaled_amax_gb300 as nv
from nvfp4_block_scaled_amax_gb300.linear import linear_layer, linear_layer_grad

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_layer_in_graphs(fmt):
    """Forward and backward captured into two graphs on one stream, replayed in turn with other inputs in place, eager calls
    on the same stream before the first replay and between."""
    T, N, K = 96, 160, 128
    def inputs(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        return [torch.randn(*s, generator=g, device="cuda").bfloat16() for s in ((T, K), (N, K), (T, N))]
    def step(x, w, dy):
        y, saved = linear_layer(x, w, format=fmt)
        return (y, *linear_layer_grad(dy, saved))
    static = inputs(0)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        graphs = []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                out = step(*static)
            graphs.append((g, out))
        for seed in range(1, 5):
            for to, v in zip(static, inputs(seed)):
                to.copy_(v)
            want = step(*static)
            for g, out in graphs:
                g.replay()
            again = step(*static)
            stream.synchronize()
            for got in (graphs[0][1], graphs[1][1], again):
                assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert nv.device_status() == 0
