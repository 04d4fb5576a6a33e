"""The C ABI of the expert-layer operators without a GPU: every bad argument is refused before any CUDA call."""
import ctypes

import pytest

from test_abi import ERR_ALIGN, ERR_CUDA, ERR_DTYPE, ERR_FLAGS, ERR_NULL, ERR_SHAPE, OK, ROW, COL, SWZ

pytestmark = pytest.mark.skipif(
    __import__("torch").cuda.is_available(),
    reason="validation-only tests with fake device addresses: run on a machine without a GPU")

X, A, B, C, D, E = (0x100000 * (i + 1) for i in range(6))  # fake, 16-byte aligned


@pytest.fixture(scope="module")
def lib():
    from nvfp4_block_scaled_amax_gb300 import _lib, build
    build.build()
    real = _lib.load()

    class Checked:
        def __getattr__(self, name):
            def call(*args):
                rc = getattr(real, name)(*args)
                if rc == ERR_CUDA:
                    pytest.fail(f"{name} accepted fake device addresses")
                return rc
            return call
    return Checked()


def test_token_rows(lib):
    rows, scratch = ctypes.c_int64(), ctypes.c_size_t()

    def ask(T, topk, experts, align):
        return lib.nvfp4_token_rows(T, topk, experts, align, ctypes.byref(rows), ctypes.byref(scratch))
    from nvfp4_block_scaled_amax_gb300 import tokens
    for T, topk, experts, align in ((1, 1, 1, 1), (5, 2, 8, 1), (1024, 2, 8, 128), (1025, 2, 8, 128), (40000, 8, 64, 16)):
        assert ask(T, topk, experts, align) == OK
        slots = T * topk
        # no assignment needs more: each expert wastes at most align - 1 rows, and members are multiples of align
        assert rows.value == (slots + experts * (align - 1)) // align * align
        assert scratch.value == (0 if slots <= tokens.SORT_CHUNK else 4 * experts * -(-slots // tokens.SORT_CHUNK))
    assert ask(0, 2, 4, 128) == OK and rows.value == 384
    for bad in ((-1, 1, 1, 1), (1, 0, 1, 1), (1, 65, 1, 1), (1, 1, 0, 1), (1, 1, 1025, 1), (1, 1, 1, 0),
                (1 << 31, 1, 1, 1), (1 << 30, 2, 1, 1), ((1 << 31) - 8, 1, 64, 128)):
        assert ask(*bad) == ERR_SHAPE
    assert lib.nvfp4_token_rows(1, 1, 1, 1, None, ctypes.byref(scratch)) == ERR_NULL


def test_sort_and_dispatch(lib):
    def sort(ids=X, T=4, topk=2, experts=8, align=1, off=A, ros=B, sor=C, rows=8, scratch=None, size=0):
        return lib.nvfp4_sort_tokens(ids, T, topk, experts, align, off, ros, sor, rows, scratch, size, None)
    assert sort(experts=0) == ERR_SHAPE
    assert sort(experts=1025) == ERR_SHAPE
    assert sort(align=0) == ERR_SHAPE
    assert sort(rows=7) == ERR_SHAPE                       # not the capacity
    assert sort(ids=None) == ERR_NULL
    assert sort(off=None) == ERR_NULL
    assert sort(sor=None) == ERR_NULL
    assert sort(ids=X + 2) == ERR_ALIGN
    assert sort(T=1025, rows=2050) == ERR_SHAPE            # two chunks need scratch
    assert sort(T=1025, rows=2050, size=64) == ERR_NULL
    assert sort(T=1025, rows=2050, scratch=D, size=63) == ERR_SHAPE

    def dispatch(x=D, dtype=0, width=64, rows=8, out=E, T=4):
        return lib.nvfp4_dispatch_tokens(x, dtype, T, width, X, 2, 8, 1, A, B, C, rows, out, None, 0, None)
    assert dispatch(dtype=2) == ERR_DTYPE
    assert dispatch(width=60) == ERR_SHAPE                 # 120-byte rows
    assert dispatch(dtype=1, width=66) == ERR_SHAPE
    assert dispatch(x=None) == ERR_NULL
    assert dispatch(out=None) == ERR_NULL
    assert dispatch(x=D + 8) == ERR_ALIGN
    assert dispatch(rows=9) == ERR_SHAPE
    assert lib.nvfp4_gather_tokens(D, 0, 4, 64, 2, B, None, 8, E, None) == ERR_NULL
    assert lib.nvfp4_gather_tokens(D, 0, 4, 64, 65, B, C, 8, E, None) == ERR_SHAPE
    assert lib.nvfp4_gather_tokens(D, 0, 4, 64, 2, B, C, 8, E + 8, None) == ERR_ALIGN


def test_combine(lib):
    def combine(rows_in=X, dtype=0, T=4, width=64, topk=2, ros=A, rows=8, w=B, y=C):
        return lib.nvfp4_combine_tokens(rows_in, dtype, T, width, topk, ros, rows, w, y, None)
    assert combine(dtype=3) == ERR_DTYPE
    assert combine(width=4) == ERR_SHAPE
    assert combine(T=-1) == ERR_SHAPE
    assert combine(rows_in=None) == ERR_NULL
    assert combine(ros=None) == ERR_NULL
    assert combine(y=None) == ERR_NULL
    assert combine(w=B + 1) == ERR_ALIGN
    assert combine(y=C + 4) == ERR_ALIGN

    def grad(dy=X, rows_in=A, ros=B, sor=C, drows=D, width=64):
        return lib.nvfp4_combine_tokens_grad(dy, rows_in, 0, 4, width, 2, ros, sor, 8, None, drows, E, None)
    assert grad(dy=None) == ERR_NULL
    assert grad(rows_in=None) == ERR_NULL
    assert grad(sor=None) == ERR_NULL
    assert grad(drows=D + 8) == ERR_ALIGN
    assert grad(width=68) == ERR_SHAPE
    most = (1 << 31) - 1
    assert lib.nvfp4_combine_tokens_grad(X, A, 0, most, 8, 1, B, C, most, None, D, E, None) == ERR_SHAPE  # CTAs of a launch


def test_fp8(lib):
    def cast(x=X, dtype=0, batch=1, M=64, N=64, br=1, dr=A, sr=B, dc=C, sc=D, flags=ROW | COL):
        return lib.nvfp4_fp8_quantize(x, dtype, batch, M, N, br, dr, sr, dc, sc, flags, None)
    assert cast(flags=0) == ERR_FLAGS
    assert cast(flags=ROW | SWZ) == ERR_FLAGS
    assert cast(dtype=2) == ERR_DTYPE
    assert cast(br=16) == ERR_SHAPE
    assert cast(N=24) == ERR_SHAPE
    assert cast(M=24) == ERR_SHAPE
    assert cast(M=-16) == ERR_SHAPE
    assert cast(batch=1 << 20, M=1 << 12) == ERR_SHAPE
    assert cast(x=None) == ERR_NULL
    assert cast(sc=None) == ERR_NULL
    assert cast(x=X + 8) == ERR_ALIGN
    assert cast(dc=C + 8) == ERR_ALIGN
    assert cast(sr=B + 2) == ERR_ALIGN

    def mm(a=X, sa=A, b=B, sb=C, br=128, M=64, N=64, K=64, out=D, dtype=0):
        return lib.nvfp4_fp8_matmul(a, sa, b, sb, br, M, N, K, out, dtype, None)
    assert mm(br=2) == ERR_SHAPE
    assert mm(K=40) == ERR_SHAPE
    assert mm(M=1 << 31) == ERR_SHAPE
    assert mm(dtype=7) == ERR_DTYPE
    assert mm(sa=None) == ERR_NULL
    assert mm(out=None) == ERR_NULL
    assert mm(a=X + 8) == ERR_ALIGN
    assert mm(sb=C + 1) == ERR_ALIGN

    def grouped(experts=4, off=E, rows=64):
        return lib.nvfp4_fp8_matmul_grouped(X, A, B, C, 128, rows, 64, 64, experts, off, D, 0, None)
    assert grouped(experts=0) == ERR_SHAPE
    assert grouped(experts=1025) == ERR_SHAPE
    assert grouped(off=None) == ERR_NULL
    assert grouped(off=E + 2) == ERR_ALIGN
    wg = lib.nvfp4_fp8_matmul_grouped_wgrad
    assert wg(X, A, B, C, 64, 64, 72, 4, E, D, 1, None) == ERR_SHAPE      # rows % 16
    assert wg(X, A, B, C, 64, 64, 64, 4, None, D, 1, None) == ERR_NULL


def test_layer_for_training_needs_the_column_wise_weights():
    import torch

    from nvfp4_block_scaled_amax_gb300.experts import expert_layer
    from nvfp4_block_scaled_amax_gb300.fp8 import FP8Operand, FP8Tensor
    w = FP8Tensor(FP8Operand(torch.zeros(2, 128, 128, dtype=torch.float8_e4m3fn), torch.ones(2, 1, 1), 128), None)
    with pytest.raises(ValueError, match="column-wise"):
        expert_layer(torch.zeros(4, 128, dtype=torch.bfloat16), w, torch.zeros(4, 1, dtype=torch.int32), torch.ones(4, 1))
