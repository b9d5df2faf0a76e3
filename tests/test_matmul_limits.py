"""Sizes that no launch can hold are refused with FP4_ERR_UNSUPPORTED before anything is launched (no
GPU needed)."""
import ctypes

import pytest

pytest.importorskip("torch")

FAKE = ctypes.c_void_p(0x1000)
BF16, E4M3 = 0, 2


@pytest.fixture(scope="module")
def L():
    from block_scaled_fp4_nvfp4_amd import _lib
    return _lib.lib()


@pytest.mark.parametrize("xd,b,m,n,k", [
    (BF16, 1, 1 << 29, 16, 128),                   # 2^32 threads quantize x's 2^29 blocks, 8 each
    (BF16, 65536, 40, 128, 128), (BF16, 65536, 4, 128, 128), (E4M3, 65536, 40, 128, 128), (E4M3, 65536, 4, 128, 128),
    (E4M3, 1, (1 << 31) - 1, 1 << 14, 128), (E4M3, 1, 300, (1 << 31) - 1, 128)])
def test_refused(L, xd, b, m, n, k):
    st = L.fp8_block_matmul(FAKE, xd, FAKE, FAKE, FAKE, b, m, n, k, FAKE, 0, FAKE, 1 << 62, None)
    assert st == -3, L.fp4_last_error()
