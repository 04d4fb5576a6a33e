"""The C ABI and the Python checks of the 4-bit operators without a GPU: bad arguments are refused before any CUDA call."""
import ctypes

import pytest
import torch

from test_abi import COL, ERR_ALIGN, ERR_CUDA, ERR_DTYPE, ERR_FLAGS, ERR_NULL, ERR_SHAPE, OK, ROW, ROWSC, SWZ

pytestmark = pytest.mark.skipif(
    torch.cuda.is_available(),
    reason="validation-only tests with fake device addresses: run on a machine without a GPU")

X, A, B, C, D, E, F, G = (0x100000 * (i + 1) for i in range(8))  # fake, 128-byte aligned


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


def operand(data=A, scale=B, amax=C, flags=0):
    from nvfp4_block_scaled_amax_gb300._lib import Operand
    return ctypes.byref(Operand(data, scale, amax, flags))


def test_operand_layout():
    from nvfp4_block_scaled_amax_gb300 import _lib, fp4
    o = _lib.Operand(1, 2, 3, 4)
    assert bytes(o)[:28] == fp4._pack(1, 2, 3, 4, 0)[:28] and len(bytes(o)) == len(fp4._pack(1, 2, 3, 4, 0))


def test_mxfp4_cast(lib):
    def cast(x=X, dtype=0, M=64, N=64, dr=A, sr=B, dc=C, sc=D, flags=ROW | COL):
        return lib.nvfp4_mxfp4_quantize(x, dtype, M, N, dr, sr, dc, sc, flags, None)
    assert cast(flags=0) == ERR_FLAGS
    assert cast(flags=ROW | 8) == ERR_FLAGS
    assert cast(dtype=2) == ERR_DTYPE
    assert cast(N=48) == ERR_SHAPE
    assert cast(M=48) == ERR_SHAPE
    assert cast(M=-32) == ERR_SHAPE
    assert cast(M=(1 << 31) - 32) == ERR_SHAPE
    assert cast(N=1 << 31) == ERR_SHAPE
    assert cast(flags=ROW | SWZ) == ERR_ALIGN              # 64 x 64
    assert cast(M=128, N=128, sr=B + 8, flags=ROW | SWZ) == ERR_ALIGN
    assert cast(x=None) == ERR_NULL
    assert cast(sr=None) == ERR_NULL
    assert cast(dc=None) == ERR_NULL
    assert cast(x=X + 8) == ERR_ALIGN
    assert cast(dr=A + 8) == ERR_ALIGN


def test_mxfp4_dequantize(lib):
    def read(data=A, scale=B, rows=4, cols=64, flags=0, out=C, dtype=0):
        return lib.nvfp4_mxfp4_dequantize(data, scale, rows, cols, flags, out, dtype, None)
    assert read(flags=ROWSC) == ERR_FLAGS
    assert read(dtype=3) == ERR_DTYPE
    assert read(cols=48) == ERR_SHAPE
    assert read(rows=-1) == ERR_SHAPE
    assert read(flags=SWZ) == ERR_ALIGN
    assert read(data=None) == ERR_NULL
    assert read(out=None) == ERR_NULL
    assert read(data=A + 4) == ERR_ALIGN
    assert read(out=C + 16) == ERR_ALIGN


def test_matmul(lib):
    def mm(a=None, b=None, block=16, M=4, N=8, K=64, out=D, dtype=0):
        return lib.nvfp4_fp4_matmul(operand() if a is None else a, operand() if b is None else b, block, M, N, K, out, dtype,
                                    None)
    assert lib.nvfp4_fp4_matmul(None, operand(), 16, 4, 8, 64, D, 0, None) == ERR_NULL
    assert mm(dtype=2) == ERR_DTYPE
    assert mm(block=8) == ERR_SHAPE
    for bad in (dict(K=48), dict(K=-32), dict(M=-1), dict(N=1 << 31), dict(M=(1 << 31) - 1), dict(K=(1 << 27) + 32),
                dict(M=1 << 28, N=1 << 28)):
        assert mm(**bad) == ERR_SHAPE
    assert mm(a=operand(flags=ROW)) == ERR_FLAGS
    assert mm(block=32) == ERR_FLAGS                       # MXFP4 with an amax
    assert mm(block=32, a=operand(amax=None, flags=ROWSC), b=operand(amax=None)) == ERR_FLAGS
    assert mm(a=operand(flags=SWZ)) == ERR_ALIGN           # 4 rows
    assert mm(M=128, K=64, a=operand(flags=SWZ)) == ERR_ALIGN
    assert mm(N=128, K=128, b=operand(scale=B + 8, flags=SWZ)) == ERR_ALIGN
    assert mm(a=operand(data=A + 8)) == ERR_ALIGN
    assert mm(b=operand(amax=C + 2)) == ERR_ALIGN
    assert mm(out=D + 8) == ERR_ALIGN
    assert mm(a=operand(data=None)) == ERR_NULL
    assert mm(b=operand(scale=None)) == ERR_NULL
    assert mm(b=operand(amax=None)) == ERR_NULL
    assert mm(out=None) == ERR_NULL


def test_expert_mlp(lib):
    n = ctypes.c_size_t()

    def size(T=4, topk=2, experts=8, H=64, I=96, block=16):
        return lib.nvfp4_expert_mlp_workspace(T, topk, experts, H, I, block, ctypes.byref(n))
    assert size() == OK and n.value > 0
    assert size(T=0) == OK
    for bad in (dict(T=-1), dict(T=1025, topk=1), dict(T=513), dict(topk=0), dict(topk=65), dict(experts=0),
                dict(experts=1025), dict(H=48), dict(I=10272), dict(H=-32), dict(block=8)):
        assert size(**bad) == ERR_SHAPE
    assert lib.nvfp4_expert_mlp_workspace(4, 2, 8, 64, 96, 16, None) == ERR_NULL
    assert size() == OK
    need = n.value

    def mlp(x=X, T=4, H=64, I=96, up=None, down=None, block=16, ids=D, gates=E, topk=2, experts=8, ws=F, size=need, y=G):
        return lib.nvfp4_expert_mlp(x, T, H, I, operand() if up is None else up, operand() if down is None else down, block,
                                    ids, gates, topk, experts, ws, size, y, None)
    assert mlp(block=64) == ERR_SHAPE
    assert mlp(H=40) == ERR_SHAPE
    assert mlp(T=600) == ERR_SHAPE
    assert mlp(size=need - 1) == ERR_SHAPE
    assert mlp(up=operand(flags=SWZ)) == ERR_FLAGS
    assert mlp(block=32) == ERR_FLAGS
    assert mlp(down=operand(amax=None)) == ERR_NULL
    for name in ("x", "ids", "gates", "ws", "y"):
        assert mlp(**{name: None}) == ERR_NULL
    assert mlp(x=X + 8) == ERR_ALIGN
    assert mlp(ws=F + 64) == ERR_ALIGN
    assert mlp(ids=D + 2) == ERR_ALIGN
    assert lib.nvfp4_expert_mlp(X, 4, 64, 96, None, operand(), 16, D, E, 2, 8, F, need, G, None) == ERR_NULL


def test_python_refuses_what_is_no_operand():
    import nvfp4_block_scaled_amax_gb300 as nv
    from nvfp4_block_scaled_amax_gb300.linear import linear_layer
    codes, scale, amax = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(16, dtype=torch.uint8), torch.ones(1)
    with pytest.raises(ValueError, match="CUDA"):
        nv.matmul_fp4(nv.FP4Operand(codes, scale, amax), nv.FP4Operand(codes, scale, amax))
    with pytest.raises(ValueError, match="dimensions"):
        nv.dequantize_fp4(nv.FP4Operand(codes[0], scale, amax))
    with pytest.raises(TypeError):
        nv.dequantize_fp4(nv.FP4Operand(codes.char(), scale, amax))
    with pytest.raises(ValueError):
        nv.quantize_mxfp4(torch.zeros(32, 32))
    with pytest.raises(ValueError):
        nv.quantize_mxfp4(torch.zeros(32))
    with pytest.raises(ValueError):
        nv.quantize_experts(torch.zeros(2, 32, 40))
    with pytest.raises(ValueError):
        linear_layer(torch.zeros(32, 32), torch.zeros(32, 32))
