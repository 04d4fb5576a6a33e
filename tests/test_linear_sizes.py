"""Sizes that the products of a 4-bit linear layer do not take are refused before anything runs (no GPU needed)."""
import pytest
import torch

from nvfp4_block_scaled_amax_gb300 import FP4Operand, FP4Tensor, NVFP4Tensor
from nvfp4_block_scaled_amax_gb300.linear import LinearSaved, linear_layer, linear_layer_grad


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("T,N,K", [(48, 64, 64), (64, 48, 64), (16, 32, 32), (33, 32, 32)])
def test_training_sizes(fmt, T, N, K):
    with pytest.raises(ValueError, match="multiples of 32"):
        linear_layer(torch.zeros(T, K), torch.zeros(N, K), format=fmt)
    with pytest.raises(ValueError, match="multiple of 32"):
        linear_layer(torch.zeros(64, 48), torch.zeros(64, 48), format=fmt)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_serving_sizes(fmt):
    """One token, or any number of rows of either, but whole blocks of what is contracted."""
    with pytest.raises(ValueError, match="multiple of 32"):
        linear_layer(torch.zeros(1, 48), torch.zeros(5, 48), format=fmt, training=False)
    with pytest.raises(ValueError, match="CUDA"):
        linear_layer(torch.zeros(1, 64), torch.zeros(5, 64), format=fmt, training=False)


def test_cast_weights():
    codes = torch.zeros(48, 32, dtype=torch.uint8)
    mx = FP4Tensor(FP4Operand(codes, codes, None, 32), FP4Operand(codes, codes, None, 32))
    nv = NVFP4Tensor(48, 64, codes, codes, torch.zeros(1), codes, codes, torch.zeros(1))
    for weight, fmt in ((mx, "mxfp4"), (nv, "nvfp4")):
        with pytest.raises(ValueError, match="multiples of 32"):
            linear_layer(torch.zeros(64, 64), weight, format=fmt)
        with pytest.raises(ValueError, match="64"):
            linear_layer(torch.zeros(64, 96), weight, format=fmt, training=False)


def test_gradient_sizes():
    codes = torch.zeros(64, 32, dtype=torch.uint8)
    mx = FP4Tensor(FP4Operand(codes, codes, None, 32), FP4Operand(codes, codes, None, 32))
    for shape in ((32, 64), (64, 32), (64,)):
        with pytest.raises(ValueError, match="dy must be"):
            linear_layer_grad(torch.zeros(shape), LinearSaved(mx, mx, "mxfp4"))
