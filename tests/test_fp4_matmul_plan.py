"""The shapes of the GPU tests reach every kernel of fp4_matmul and fp4_matmul_grad: a change of the plan's rules that
takes one out of their reach fails here (no GPU needed)."""
import ctypes

import pytest

pytest.importorskip("torch")

from fp4_shapes import FEW, TILES  # noqa: E402

FMT, DT = {"nvfp4": 0, "mxfp4": 1}, {"bf16": 0, "f32": 1}


@pytest.fixture(scope="module")
def plan():
    from block_scaled_fp4_nvfp4_amd import _lib
    f = _lib.lib().fp4_matmul_plan
    f.argtypes = [ctypes.c_int] * 3 + [ctypes.c_int64] * 4 + [ctypes.POINTER(ctypes.c_int * 5)]

    def ask(fmt, x, grad, b, m, n, k):
        p = (ctypes.c_int * 5)()
        assert f(FMT[fmt], DT[x], grad, b, m, n, k, ctypes.byref(p)) == 0
        return dict(zip(("few", "rows", "outputs", "shared", "copied"), p))
    return ask


def test_every_tile(plan):
    reached = set()
    for fmt, x, grad, b, m, n, k in TILES:
        p = plan(fmt, x, grad, b, m, n, k)
        assert not p["few"], (fmt, x, grad, m, n, k)
        pairs = fmt == "nvfp4" and k % 32 == 0  # a thread's two scales as one load
        reached |= {(p["rows"], x, grad, "shared" if p["shared"] > 1 else "whole"), (p["rows"], x, grad, fmt), (p["rows"], grad, fmt, pairs)}
    for x in ("bf16", "f32"):
        for grad in (False, True):
            for rows in (16, 64, 128, 256):
                assert {(rows, x, grad, "nvfp4"), (rows, x, grad, "mxfp4"), (rows, x, grad, "shared")} <= reached, (rows, x, grad)
            for rows in (64, 128, 256):
                assert (rows, x, grad, "whole") in reached, (rows, x, grad)
    for rows in (16, 128, 256):
        for grad in (False, True):
            assert {(rows, grad, "nvfp4", True), (rows, grad, "nvfp4", False)} <= reached, (rows, grad)
    assert {(32, "bf16", False, "mxfp4"), (32, "f32", False, "nvfp4"), (32, "f32", False, "mxfp4"), (32, "f32", True, "nvfp4"), (32, "f32", True, "mxfp4")} <= reached


def test_every_block_of_few_rows(plan):
    reached = set()
    for fmt, x, m, n, k in FEW:
        p = plan(fmt, x, False, 1, m, n, k)
        assert p["few"], (fmt, x, m, n, k)
        steps = (k + 255) // 256
        waves = {("bf16", 1): (8, 8, 7, 7), ("bf16", 2): (8, 7), ("bf16", 4): (7,), ("f32", 1): (7, 7)}[x, p["few"]]  # for 1, 2, 4 steps a wave
        each = next(u for u in (1, 2, 4) if -(-steps // u) <= waves[u - 1])
        reached.add((fmt, x, p["few"], each, k % (64 if fmt == "nvfp4" else 128) == 0))
    for fmt in ("nvfp4", "mxfp4"):
        for dma in (False, True):
            for x, blocks, each in (("bf16", 1, 1), ("bf16", 1, 2), ("bf16", 1, 4), ("bf16", 2, 1), ("bf16", 2, 2), ("bf16", 4, 1), ("f32", 1, 1), ("f32", 1, 2)):
                assert (fmt, x, blocks, each, dma) in reached, (fmt, x, blocks, each, dma)
