"""Sizes of fp4_matmul and fp4_matmul_grad that no launch can hold are refused with FP4_ERR_UNSUPPORTED, by the workspace
query too and before anything is launched (no GPU needed: a launch would fail with FP4_ERR_HIP here)."""
import ctypes

import pytest

pytest.importorskip("torch")

FAKE = ctypes.c_void_p(0x1000)
BF16, F32 = 0, 1


@pytest.fixture(scope="module")
def L():
    from block_scaled_fp4_nvfp4_amd import _lib
    return _lib.lib()


# (type, batch, m, length of the sum, outputs): tiles of aligned rows, of rows that are copied or split first; rows to copy
@pytest.mark.parametrize("xd,b,m,c,o", [(BF16, 1, 1 << 30, 64, 1024), (BF16, 1, 1 << 27, 80, 1 << 17), (F32, 1, 1 << 27, 64, 1 << 17), (BF16, 1, 300, 64, (1 << 31) - 32),
                                        (BF16, 1, 1 << 28, 80, 32), (BF16, 1, (1 << 28) - 1, 80, 32), (F32, 16, 1 << 25, 64, 32), (F32, 1, (1 << 29) - 1, 64, 32)])
@pytest.mark.parametrize("grad", [False, True], ids=["product", "gradient"])
def test_refused_before_any_work(L, xd, b, m, c, o, grad):
    n, k = (c, o) if grad else (o, c)
    name = "fp4_matmul_grad" if grad else "fp4_matmul"
    size = ctypes.c_size_t()
    if grad and k > 1 << 26:
        pytest.skip("k above 2^26 is refused anyway")
    assert getattr(L, name + "_workspace_size")(0, xd, b, m, n, k, ctypes.byref(size)) == -3
    assert getattr(L, name)(0, FAKE, xd, FAKE, FAKE, FAKE, b, m, n, k, FAKE, 0, FAKE, 1 << 62, None) == -3, L.fp4_last_error()


@pytest.mark.parametrize("grad", [False, True], ids=["product", "gradient"])
def test_large_sizes_are_planned(L, grad):
    """Just below: the query answers."""
    size = ctypes.c_size_t()
    query = L.fp4_matmul_grad_workspace_size if grad else L.fp4_matmul_workspace_size
    for m, c, o in ((1 << 24, 64, 1024), (1 << 27, 80, 32), ((1 << 28) - 2048, 80, 32)):
        assert query(0, BF16, 1, m, c if grad else o, o if grad else c, ctypes.byref(size)) == 0, L.fp4_last_error()
