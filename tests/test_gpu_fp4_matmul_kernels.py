"""Every kernel of fp4_matmul and fp4_matmul_grad against float64 (tolerances: head_util.check_product), with scales at any
address, operands that end where NaN and 0xFF begin, results inside a canary."""
import pytest

from gpu_util import gpu_ok, print_case, torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_ok(), reason="needs a GPU")]

from fp4_shapes import FEW, TILES  # noqa: E402
from head_util import check_product, gen, raw_weight, w64  # noqa: E402

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _inside(t, fill, off=0, room=4096):
    """A copy of t inside memory of `fill`, `off` values behind an aligned address."""
    big = torch.full((t.numel() + 2 * room,), fill, dtype=t.dtype, device="cuda")
    part = big[room + off:room + off + t.numel()].view(t.shape)
    part.copy_(t)
    return big, part


def _check(fmt, x, grad, b, m, n, k, offs):
    import block_scaled_fp4_nvfp4_amd as fp
    print_case(f"{'grad' if grad else 'matmul'} {fmt} b={b} m={m} n={n} k={k} {x}")
    g = gen(m + n + k)
    c, o = (n, k) if grad else (k, n)
    xv = (torch.randn(b, m, c, device="cuda", generator=g) * torch.exp(torch.randn(b, m, 1, device="cuda", generator=g))).to(DT[x])
    w = raw_weight(g, fmt, b, n, k)
    W = w64(w, fmt)
    W = W if grad else W.transpose(-1, -2)
    _, xi = _inside(xv, float("nan"))
    _, codes = _inside(w["codes"], 0xFF)
    call, first = fp.fp4_matmul_grad if grad else fp.fp4_matmul, None
    for i, off in enumerate(offs):
        out_type = torch.bfloat16 if i == 1 else torch.float32
        _, scales = _inside(w["scales"], 0x7F if fmt == "nvfp4" else 0xFF, off)
        res, out = _inside(torch.zeros(b, m, o, dtype=out_type, device="cuda"), 7.0)
        call(xi, {**w, "codes": codes, "scales": scales}, fmt, out_dtype=out_type, out=out)
        assert bool((res[:4096] == 7.0).all()) and bool((res[4096 + out.numel():] == 7.0).all())
        if first is None:
            first = out
            check_product(out, xv, W, 3 if x == "f32" else 1)
        else:  # the same sums, whichever way the scales are loaded
            assert torch.equal(out, first.to(out_type))


@pytest.mark.parametrize("fmt,x,grad,b,m,n,k", TILES)
def test_tiles(fmt, x, grad, b, m, n, k):
    _check(fmt, x, grad, b, m, n, k, (0, 0, 1, 2, 3))


@pytest.mark.parametrize("fmt,x,m,n,k", FEW)
def test_few_rows(fmt, x, m, n, k):
    """(Scales that do not start at a multiple of 4 bytes come without DMA, in the same order of sums.)"""
    _check(fmt, x, False, 1, m, n, k, (0, 0, 1, 2))


@pytest.mark.parametrize("fmt,x,grad,b,m,n,k", TILES)
def test_bits_repeat(fmt, x, grad, b, m, n, k):
    """The same call again and again, other work between, gives the same bits."""
    import block_scaled_fp4_nvfp4_amd as fp
    print_case(f"repeat {'grad' if grad else 'matmul'} {fmt} b={b} m={m} n={n} k={k} {x}")
    g = gen(m)
    xv = torch.randn(b, m, n if grad else k, device="cuda", generator=g).to(DT[x])
    w = raw_weight(g, fmt, b, n, k)
    call = fp.fp4_matmul_grad if grad else fp.fp4_matmul
    first = call(xv, w, fmt, out_dtype=torch.float32)
    for _ in range(4):
        xv * 2
        assert torch.equal(call(xv, w, fmt, out_dtype=torch.float32), first)
