"""The product kernels' wait: it ends by itself on a barrier that nobody signals, reports it, and leaves the context
usable."""
import ctypes
import os
import subprocess
import time

import pytest
import torch

from nvfp4_block_scaled_amax_gb300 import build as nvbuild

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def lib():
    os.makedirs(os.path.join(HERE, "_build"), exist_ok=True)
    out = os.path.join(HERE, "_build", "libfp8selftest.so")
    subprocess.check_call([nvbuild.nvcc(), *nvbuild.NVCC_FLAGS, "-shared", "-o", out,
                           os.path.join(HERE, "fp8_selftest.cu")])
    L = ctypes.CDLL(out)
    L.selftest_product_wait.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p]
    return L


@pytest.mark.parametrize("signal", [1, 0])
def test_wait_is_bounded(lib, signal):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    result = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    t0 = time.monotonic()
    assert lib.selftest_product_wait(status.data_ptr(), signal, result.data_ptr()) == 0
    took = time.monotonic() - t0
    assert result.item() == signal
    assert status.item() == (0 if signal else 1)
    # 2^19 tries of at most some thousand cycles each: seconds at the very most
    assert took < 20.0
    assert float((torch.ones(8, device="cuda") * 2).sum()) == 16.0
