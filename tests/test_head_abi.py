"""fp4_matmul, fp4_matmul_grad, token_logprobs and token_logprobs_grad refuse bad
arguments on the host (no GPU needed: every call here returns before any HIP
call), and their Python bindings check shapes, types and devices before that."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

FAKE, ODD, ODD2 = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1004), ctypes.c_void_p(0x1001)


@pytest.fixture(scope="module")
def L():
    from block_scaled_fp4_nvfp4_amd import _lib
    return _lib.lib()


@pytest.fixture(params=[False, True], ids=["product", "gradient"])
def mm(request, L):
    f = L.fp4_matmul_grad if request.param else L.fp4_matmul

    def call(fmt=0, x=FAKE, xd=0, w=FAKE, ws=FAKE, ts=FAKE, b=1, m=4, n=128, k=256, y=FAKE, yd=0, wk=None, wb=0):
        return f(fmt, x, xd, w, ws, ts, b, m, n, k, y, yd, wk, wb, None)
    call.grad = request.param
    call.size = L.fp4_matmul_grad_workspace_size if request.param else L.fp4_matmul_workspace_size
    return call


def test_product_refusals(mm, L):
    assert mm(fmt=6) == -1 and mm(fmt=-1) == -1
    assert mm(fmt=2) == -3 and mm(fmt=3) == -3 and mm(fmt=5) == -3   # other formats
    assert mm(xd=2) == -1 and mm(xd=7) == -1 and mm(yd=2) == -1
    assert mm(k=24) == -2 and mm(fmt=1, k=48) == -2
    assert b"multiple" in L.fp4_last_error()
    assert (mm(n=0) if mm.grad else mm(k=0)) == -2                    # sums of nothing
    for kw in ({"m": -1}, {"n": -1}, {"b": -1}, {"k": -16}):
        assert mm(**kw) == -2
    for kw in ("x", "w", "ws", "y", "ts"):
        assert mm(**{kw: None}) == -1, kw
    assert mm(fmt=1, ts=None, y=None) == -1                           # MXFP4 needs no tensor scale, but a result
    assert mm(x=ODD) == -1 and mm(w=ODD) == -1 and mm(ts=ODD2) == -1
    assert mm(y=ODD2) == -1 and mm(yd=1, y=ctypes.c_void_p(0x1002)) == -1
    assert mm(m=1 << 31) == -3 and mm(n=1 << 40) == -3 and mm(b=65536) == -3
    assert mm(**({"n": (1 << 22) + 64} if mm.grad else {"k": (1 << 22) + 64})) == -3
    assert mm(b=1 << 15, m=1 << 20, n=64, k=1 << 20) == -3


def test_product_empty(mm):
    assert mm(b=0) == 0 and mm(m=0, x=None) == 0
    assert (mm(k=0, w=None) if mm.grad else mm(n=0, w=None)) == 0


def test_product_workspace(mm):
    sz = ctypes.c_size_t()
    ask = lambda *a: mm.size(*a, ctypes.byref(sz))  # noqa: E731
    assert mm.size(0, 0, 1, 4, 128, 256, None) == -1
    assert ask(0, 1, 3, 200, 128, 256) == 0 and sz.value >= 3 * 200 * 6 * (128 if mm.grad else 256)  # f32: three terms
    need = sz.value
    bad = dict(xd=1, b=3, m=200, n=128, k=256)
    assert mm(**bad) == -4 and mm(**bad, wk=FAKE, wb=need - 1) == -4
    assert mm(**bad, wk=ODD, wb=1 << 26) == -1
    if not mm.grad:
        assert ask(0, 1, 3, 70, 128, 256) == 0 and sz.value == 0                                     # few rows are split inside the product
    assert ask(0, 0, 1, 70, 100, 272) == 0 and sz.value >= 70 * 2 * (128 if mm.grad else 320)      # rows padded to 64
    assert ask(9, 0, 1, 4, 128, 256) == -1 and ask(0, 0, 1, 4, 128, 255) == -2


def _lp(L, logits=FAKE, dt=0, T=4, V=100, stride=100, targets=FAKE, temp=1.0, top=0, lp=FAKE, rk=FAKE, ids=None, tl=None, st=FAKE, wk=None, wb=0):
    return L.token_logprobs(logits, dt, T, V, stride, targets, temp, top, lp, rk, ids, tl, st, wk, wb, None)


def _lg(L, logits=FAKE, dt=0, T=4, V=100, stride=100, targets=FAKE, temp=1.0, st=FAKE, gl=FAKE, ge=None, d=FAKE, ds=100):
    return L.token_logprobs_grad(logits, dt, T, V, stride, targets, temp, st, gl, ge, d, ds, None)


@pytest.mark.parametrize("f", [_lp, _lg], ids=["logprobs", "gradient"])
def test_logprob_refusals(L, f):
    assert f(L, dt=2) == -1 and f(L, dt=-1) == -1
    assert f(L, T=-1) == -2 and f(L, V=0) == -2 and f(L, stride=99) == -2
    assert f(L, V=1 << 30, stride=1 << 30, **({"ds": 1 << 30} if f is _lg else {})) == -3
    assert f(L, T=1 << 31) == -3 and f(L, T=1 << 20, stride=1 << 39) == -3
    for t in (0.0, -1.0, float("inf"), float("nan")):
        assert f(L, temp=t) == -1, t
    assert f(L, logits=None) == -1 and f(L, targets=None) == -1
    assert f(L, logits=ODD2) == -1 and f(L, dt=1, logits=ctypes.c_void_p(0x1002)) == -1 and f(L, targets=ODD2) == -1 and f(L, st=ODD2) == -1
    assert f(L, T=0, logits=None) == 0


@pytest.mark.parametrize("f", [_lp, _lg], ids=["logprobs", "gradient"])
def test_logprob_least_temperature(L, f):
    assert f(L, temp=2.0 ** -101) == -1 and f(L, temp=1e-45) == -1   # far below, 1 / T overflows
    assert f(L, temp=2.0 ** -100, T=0) == 0 and f(L, temp=3.4e38, T=0) == 0


def test_logprob_refusals_of_outputs(L):
    assert _lp(L, top=65) == -1 and _lp(L, top=-1) == -1
    assert _lp(L, top=3) == -1 and _lp(L, top=3, ids=FAKE) == -1 and _lp(L, top=3, tl=FAKE) == -1
    assert _lp(L, lp=ODD2) == -1 and _lp(L, rk=ODD2) == -1 and _lp(L, top=1, ids=ODD2, tl=FAKE) == -1
    assert _lg(L, st=None) == -1 and _lg(L, d=None) == -1 and _lg(L, ds=99) == -2
    assert _lg(L, d=ODD2) == -1 and _lg(L, gl=ODD2) == -1 and _lg(L, ge=ODD2) == -1
    assert L.token_logprobs_workspace_size(0, 4, 100, 0, None) == -1
    assert L.token_logprobs_workspace_size(0, 4, 100, 65, ctypes.byref(ctypes.c_size_t())) == -1


def _record(n=32, k=64, fmt="nvfp4"):
    return {"codes": torch.zeros(n, k // 2, dtype=torch.uint8), "scales": torch.zeros(n, k // (16 if fmt == "nvfp4" else 32), dtype=torch.uint8),
            "tensor_scale": torch.ones(1)}


def test_binding_of_products():
    import block_scaled_fp4_nvfp4_amd as fp
    x = torch.zeros(3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensors"):
        fp.fp4_matmul(x, _record(), "nvfp4")
    with pytest.raises(ValueError, match="nvfp4 or mxfp4"):
        fp.fp4_matmul(x, _record(), "mxfp8")
    with pytest.raises(TypeError):
        fp.fp4_matmul(x.half(), _record(), "nvfp4")
    with pytest.raises(TypeError):
        fp.fp4_matmul(x, _record(), "nvfp4", out_dtype=torch.float16)
    with pytest.raises(TypeError):
        fp.fp4_matmul(x, {**_record(), "tensor_scale": None}, "nvfp4")
    with pytest.raises(TypeError):
        fp.fp4_matmul(x, {**_record(), "scales": torch.zeros(32, 4)}, "nvfp4")
    with pytest.raises(ValueError, match="do not match"):
        fp.fp4_matmul(x[:, :32].contiguous(), _record(), "nvfp4")
    with pytest.raises(ValueError, match="do not match"):
        fp.fp4_matmul_grad(x, _record(), "nvfp4")       # dy has n columns
    with pytest.raises(ValueError, match="scales"):
        fp.fp4_matmul(x, {**_record(), "scales": torch.zeros(32, 3, dtype=torch.uint8)}, "nvfp4")
    with pytest.raises(ValueError, match="scales"):
        fp.fp4_matmul(x, _record(fmt="mxfp4"), "nvfp4")
    with pytest.raises(ValueError):
        fp.fp4_matmul(x[0], _record(), "nvfp4")


def test_binding_of_logprobs():
    import block_scaled_fp4_nvfp4_amd as fp
    with pytest.raises(ValueError, match="device tensor"):
        fp.token_logprobs(torch.zeros(2, 10), None)
    with pytest.raises(ValueError, match="device tensor"):
        fp.token_logprobs_grad(torch.zeros(2, 10), None, torch.zeros(2, 3), None)
