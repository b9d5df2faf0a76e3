"""fp8_block_matmul refuses bad arguments on the host (no GPU needed: every
call here returns before any HIP call), and its Python binding checks shapes,
types and devices before it calls the library."""
import ctypes

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def L():
    from block_scaled_fp4_nvfp4_amd import _lib
    return _lib.lib()


FAKE, ODD = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008)


def _call(L, x=FAKE, xd=2, xs=FAKE, w=FAKE, ws=FAKE, b=1, m=4, n=128, k=256, y=FAKE, yd=0, wk=None, wb=0):
    return L.fp8_block_matmul(x, xd, xs, w, ws, b, m, n, k, y, yd, wk, wb, None)


def test_refusals(L):
    assert _call(L, xd=3) == -1 and _call(L, yd=2) == -1          # unknown dtypes
    assert _call(L, k=192) == -2 and _call(L, k=0) == -2            # 128-blocks
    assert b"128" in L.fp4_last_error() or b"k is 0" in L.fp4_last_error()
    assert _call(L, m=-1) == -2 and _call(L, n=-1) == -2 and _call(L, b=-1) == -2
    for kw in ("x", "w", "ws", "y", "xs"):
        assert _call(L, **{kw: None}) == -1, kw
    assert _call(L, x=ODD) == -1 and _call(L, w=ODD) == -1           # 16-byte alignment
    assert _call(L, y=ctypes.c_void_p(0x1001)) == -1 and _call(L, yd=1, y=ctypes.c_void_p(0x1002)) == -1
    assert _call(L, m=1 << 31) == -3 and _call(L, n=1 << 40) == -3
    assert _call(L, b=1 << 20, m=1 << 20, n=128, k=1 << 20) == -3
    assert _call(L, b=1 << 20) == -3                                 # more matrices than a grid holds


def test_workspace(L):
    sz = ctypes.c_size_t()
    size = L.fp8_block_matmul_workspace_size
    assert size(2, 1, 4, 128, 256, ctypes.byref(sz)) == 0 and sz.value == 0
    assert size(0, 3, 70, 128, 256, ctypes.byref(sz)) == 0 and sz.value >= 3 * 70 * (256 + 4 * 2)
    assert size(0, 3, 5, 128, 256, ctypes.byref(sz)) == 0 and sz.value == 0  # few rows are quantized inside the product
    assert size(0, 1, 4, 128, 256, None) == -1
    # a workspace that is missing, too small or misaligned is refused before any launch; 33 rows take one
    assert size(0, 1, 33, 128, 256, ctypes.byref(sz)) == 0
    assert _call(L, xd=0, m=33) == -4
    assert _call(L, xd=1, m=33, wk=FAKE, wb=sz.value - 1) == -4
    assert _call(L, xd=0, m=33, wk=ODD, wb=1 << 20) == -1


def test_empty_is_a_no_op(L):
    for kw in (dict(m=0), dict(n=0), dict(b=0)):
        assert _call(L, x=None, w=None, xs=None, ws=None, y=None, **kw) == 0


def test_binding_refusals():
    """CPU tensors and mismatched records never reach the library."""
    import block_scaled_fp4_nvfp4_amd as fp
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    w = {"codes": torch.zeros(130, 256, dtype=torch.uint8), "scales": torch.zeros(2, 2)}
    with pytest.raises(ValueError):
        fp.fp8_matmul(x, w)                                   # not on a device
    with pytest.raises(ValueError):
        fp.fp8_matmul(x[:, :128], w)                          # K differs
    with pytest.raises(ValueError):
        fp.fp8_matmul(x, dict(w, scales=torch.zeros(1, 2)))   # scale rows for 128 of 130 outputs
    with pytest.raises(ValueError):
        fp.fp8_matmul(torch.zeros(2, 4, 256, dtype=torch.bfloat16), w)  # batch differs
    with pytest.raises(TypeError):
        fp.fp8_matmul(x.half(), w)
    with pytest.raises(TypeError):
        fp.fp8_matmul(x, dict(w, codes=w["codes"].to(torch.int8)))
    with pytest.raises(TypeError):
        fp.fp8_matmul({"codes": torch.zeros(4, 256, dtype=torch.uint8), "scales": torch.zeros(4, 2, dtype=torch.float64)}, w)
    with pytest.raises(TypeError):
        fp.fp8_matmul(x, w, out_dtype=torch.float16)
