"""fp4_matmul and fp4_matmul_grad against float64 products of the weights' exact
values (tolerances: head_util.check_product)."""
import pytest

from gpu_util import gpu_ok, print_case, torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_ok(), reason="needs a GPU")]

from head_util import BLOCK, check_product, gen, raw_weight, w64  # noqa: E402

FMTS = ["nvfp4", "mxfp4"]
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _m():
    import block_scaled_fp4_nvfp4_amd as m
    return m


def _call(grad):
    return _m().fp4_matmul_grad if grad else _m().fp4_matmul


def _x(g, b, m, c, dtype):
    return (torch.randn(b, m, c, device="cuda", generator=g) * torch.exp(torch.randn(b, m, 1, device="cuda", generator=g))).to(dtype)


def _wt(w, fmt, grad):
    v = w64(w, fmt)
    return v if grad else v.transpose(-1, -2)


# (batch, m, n, k in blocks)
SIZES = [(1, 1, 1, 1), (1, 1, 16, 2), (1, 2, 17, 3), (1, 15, 130, 5), (1, 16, 128, 80), (1, 17, 257, 40), (1, 33, 64, 81), (1, 63, 1000, 16),
         (1, 64, 127, 31), (1, 65, 640, 4), (1, 100, 129, 72), (3, 7, 48, 8), (2, 129, 300, 17), (1, 255, 513, 24), (1, 256, 256, 64),
         (1, 300, 2560, 40), (5, 70, 512, 8), (1, 513, 1290, 80), (1, 1, 4099, 320), (1, 9, 250, 324), (1, 700, 40, 160), (1, 16, 5000, 80),
         (1, 1100, 2050, 33), (1, 5, 3, 640)]


@pytest.mark.parametrize("b,m,n,kb", SIZES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("grad", [False, True], ids=["product", "gradient"])
@pytest.mark.parametrize("x,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
def test_sizes(b, m, n, kb, fmt, grad, x, out):
    k = kb * BLOCK[fmt]
    print_case(f"{'grad' if grad else 'matmul'} {fmt} b={b} m={m} n={n} k={k} {x}->{out}")
    g = gen(b * 7 + m * 3 + n + k)
    xv, w = _x(g, b, m, n if grad else k, DT[x]), raw_weight(g, fmt, b, n, k)
    y = _call(grad)(xv, w, fmt, out_dtype=DT[out])
    assert y.shape == (b, m, k if grad else n) and y.dtype == DT[out]
    check_product(y, xv, _wt(w, fmt, grad), 3 if x == "f32" else 1)
    assert torch.equal(y, _call(grad)(xv, w, fmt, out_dtype=DT[out]))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("grad", [False, True], ids=["product", "gradient"])
@pytest.mark.parametrize("m", [1, 16, 50, 200])
def test_library_weights_two_dimensions_and_out(fmt, grad, m):
    """Records as quantize() makes them; [M, K] operands; results into `out`, with and without a workspace."""
    print_case(f"library weights {fmt} grad={grad} m={m}")
    fp, n, k = _m(), 200, 448
    g = gen(m)
    q = fp.quantize(torch.randn(n, k, device="cuda", generator=g) * 0.02, fmt)
    x = _x(g, 1, m, n if grad else k, torch.bfloat16)[0]
    w = {name: None if v is None else v[None] if name != "tensor_scale" else v for name, v in q.items() if name != "m4"}
    y = _call(grad)(x, q, fmt, out_dtype=torch.float32)
    check_product(y[None], x[None], _wt(w, fmt, grad), 1)
    out = torch.full_like(y, float("nan"))
    size = fp.fp4_matmul_workspace_size(torch.bfloat16, 1, m, n, k, fmt, grad)
    space = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") if size else None
    assert _call(grad)(x, q, fmt, out_dtype=torch.float32, out=out, workspace=space) is out
    assert torch.equal(out, y)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("grad", [False, True], ids=["product", "gradient"])
@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,kb", [(3, 70, 9), (16, 600, 40), (90, 133, 24), (300, 520, 12)])
def test_exact_sums(fmt, grad, x, m, n, kb):
    """Small whole numbers, scales of few bits: every partial sum is exact in f32, so the result is too.
    The gradient equals differences of the product, which is linear."""
    k = kb * BLOCK[fmt]
    print_case(f"exact {fmt} grad={grad} {x} m={m} n={n} k={k}")
    g = gen(m + n)
    w = raw_weight(g, fmt, 1, n, k)
    if fmt == "nvfp4":  # 0.5 .. 1.875
        w["scales"] = torch.randint(0x30, 0x40, w["scales"].shape, dtype=torch.uint8, device="cuda", generator=g)
        w["tensor_scale"] = torch.tensor([2.0 ** -9], device="cuda")
    else:
        w["scales"] = torch.randint(126, 129, w["scales"].shape, dtype=torch.uint8, device="cuda", generator=g)
    xv = torch.randint(-4, 5, (1, m, n if grad else k), device="cuda", generator=g).to(DT[x])
    y = _call(grad)(xv, w, fmt, out_dtype=torch.float32)
    assert torch.equal(y.double(), torch.matmul(xv.double(), _wt(w, fmt, grad).contiguous()))
    if grad:  # d sum(dy * y) / dx_j by a difference of step 1
        j = k // 2
        e = torch.zeros(1, m, k, device="cuda", dtype=DT[x])
        e[..., j] = 1
        d = _m().fp4_matmul(e, w, fmt, out_dtype=torch.float32) - _m().fp4_matmul(-e, w, fmt, out_dtype=torch.float32)
        assert torch.equal((d.double() * xv.double()).sum(-1) / 2, y[..., j].double())


@pytest.mark.parametrize("m", [2, 40, 150])
def test_f32_values_need_all_their_bits(m):
    """f32 x = 1 + 2^-23 times a code of 1 on one column: the result keeps x's last bit; the largest f32 stays finite."""
    print_case(f"f32 bits m={m}")
    fp, n, k = _m(), 48, 64
    w = {"codes": torch.full((1, n, k // 2), 0x22, dtype=torch.uint8, device="cuda"),
         "scales": torch.full((1, n, k // 32), 127, dtype=torch.uint8, device="cuda")}
    x = torch.zeros(1, m, k, device="cuda")
    x[..., 5] = 1 + 2.0 ** -23
    x[0, 0, 5] = torch.finfo(torch.float32).max
    x[0, 1, 5] = 2.0 ** -126
    y = fp.fp4_matmul(x, w, "mxfp4", out_dtype=torch.float32)
    assert torch.equal(y, x[..., 5:6].expand(1, m, n))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m", [1, 16, 70])
def test_every_code_and_scale(fmt, m):
    """Each of the 16 codes under each of the scale bytes, as one-hot rows of x pick them out: the result is
    the weight as fp4_dequantize has it (an infinity or NaN among it stays in its own column)."""
    print_case(f"codes {fmt} m={m}")
    fp, B = _m(), BLOCK[fmt]
    n, k = 256, B
    codes = torch.arange(B, device="cuda") % 16
    packed = (codes[0::2] | (codes[1::2] << 4)).to(torch.uint8).expand(1, n, -1).contiguous()
    scales = torch.arange(256, device="cuda").to(torch.uint8).reshape(1, n, 1).contiguous()
    w = {"codes": packed, "scales": scales, "tensor_scale": torch.tensor([0.75], device="cuda")}
    ref = w64(w, fmt)[0].float()  # [n, k]; f32: beyond its range infinite
    if fmt == "mxfp4":
        ref[255] = float("nan")
    for first in range(0, 16, m):
        x = torch.zeros(m, k, device="cuda", dtype=torch.bfloat16)
        for i in range(m):
            x[i, (first + i) % 16] = 1
        y = fp.fp4_matmul(x, w, fmt, out_dtype=torch.float32)
        finite = torch.isfinite(ref).all(1)  # 0 times an infinity elsewhere in the row is NaN
        for i in range(m):
            assert torch.equal(y[i][finite], ref[finite][:, (first + i) % 16]), (first, i)
        assert not bool(torch.isfinite(y[:, ~finite]).any())
    dy = torch.zeros(1, n, device="cuda", dtype=torch.bfloat16)
    for row in (1, 60, 120, 200):  # the gradient of one output is that row of W
        dy.zero_()
        dy[0, row] = 1
        ww = {**w, "scales": torch.where(torch.isfinite(ref).all(1).reshape(1, n, 1), scales, torch.ones_like(scales))}
        dx = fp.fp4_matmul_grad(dy, ww, fmt, out_dtype=torch.float32)
        assert torch.equal(dx[0], w64(ww, fmt)[0, row].float())


@pytest.mark.parametrize("S", [0.0, 2.0 ** -149, 2.0 ** -126, 1e-30, 3.3e30, 1.7e38])
@pytest.mark.parametrize("m", [1, 16, 100])
@pytest.mark.parametrize("grad", [False, True], ids=["product", "gradient"])
def test_tensor_scales_at_the_edges(S, m, grad):
    """x of about 1 / S: sums and results stay of size 1, whatever the tensor scale."""
    print_case(f"tensor scale {S} m={m} grad={grad}")
    n, k = 96, 256
    g = gen(m)
    w = raw_weight(g, "nvfp4", 1, n, k)
    w["scales"] = torch.randint(0x30, 0x50, w["scales"].shape, dtype=torch.uint8, device="cuda", generator=g)
    w["tensor_scale"] = torch.tensor([S], device="cuda")
    size = min(max(1 / max(S, 1e-37), 1e-37), 1e37)
    xv = torch.randn(1, m, n if grad else k, device="cuda", generator=g) * size
    if S == 2.0 ** -149:
        xv = xv * 1e7  # x up to f32's largest values
        xv = xv.clamp(-1e37, 1e37)
    for dtype in (torch.bfloat16, torch.float32):
        x = xv.to(dtype)
        y = _call(grad)(x, w, "nvfp4", out_dtype=torch.float32)
        e = torch.matmul(x.double(), _wt(w, "nvfp4", grad).contiguous())
        p = torch.matmul(x.double().abs(), _wt(w, "nvfp4", grad).abs().contiguous())
        # f32's smallest step on top: results of tiny tensor scales are subnormal.  f32 x is three bf16 terms of 8 bits
        # each; bf16's smallest step is 2^-133, so that the last one loses less than that of an x below 2^-109
        lost = 2.0 ** -133 * _wt(w, "nvfp4", grad).abs().sum(1, keepdim=True) if dtype == torch.float32 else 0.0
        assert bool(((y.double() - e).abs() <= (3 * x.shape[-1] + 16) * 2.0 ** -23 * p + 2.0 ** -126 + lost).all())


@pytest.mark.parametrize("m", [3, 16, 40, 260])
@pytest.mark.parametrize("grad", [False, True], ids=["product", "gradient"])
def test_rows_and_matrices_keep_their_bits(m, grad):
    """A row's result does not depend on the other rows (NaN among them), a matrix's not on the others."""
    print_case(f"rows m={m} grad={grad}")
    n, k = 333, 320
    g = gen(m)
    w = raw_weight(g, "nvfp4", 2, n, k)
    x = _x(g, 2, m, n if grad else k, torch.bfloat16)
    y = _call(grad)(x, w, "nvfp4")
    z = x.clone()
    z[0, 1:] = float("nan")
    z[1] = 3e38
    other = {key: v.clone() for key, v in w.items()}
    other["scales"][1] = 0x7E
    y2 = _call(grad)(z, other, "nvfp4")
    assert torch.equal(y[0, 0], y2[0, 0])
    assert bool(torch.isnan(y2[0, 1:]).all())


@pytest.mark.parametrize("grad", [False, True], ids=["product", "gradient"])
@pytest.mark.parametrize("m,n,k", [(1, 250, 2560), (16, 77, 272), (33, 129, 400), (130, 257, 96)])
def test_nothing_outside_is_read_or_written(grad, m, n, k):
    """Operands inside larger tensors of NaN and 0xFF, the result inside a canary."""
    print_case(f"guard m={m} n={n} k={k} grad={grad}")
    g = gen(n)
    w = raw_weight(g, "nvfp4", 1, n, k)
    c, o = (n, k) if grad else (k, n)
    x = _x(g, 1, m, c, torch.bfloat16)
    big = torch.full((m * c + 4096,), float("nan"), dtype=torch.bfloat16, device="cuda")
    xv = big[2048:2048 + m * c].view(1, m, c)
    xv.copy_(x)
    ww = {"tensor_scale": w["tensor_scale"]}
    for key in ("codes", "scales"):
        room = torch.full((w[key].numel() + 8192,), 0xFF, dtype=torch.uint8, device="cuda")
        ww[key] = room[4096:4096 + w[key].numel()].view(w[key].shape)
        ww[key].copy_(w[key])
    res = torch.full((m * o + 2048,), 7.0, device="cuda")
    out = res[1024:1024 + m * o].view(1, m, o)
    _call(grad)(xv, ww, "nvfp4", out_dtype=torch.float32, out=out)
    assert bool((res[:1024] == 7.0).all()) and bool((res[1024 + m * o:] == 7.0).all())
    check_product(out, x, _wt(w, "nvfp4", grad), 1)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("grad", [False, True], ids=["product", "gradient"])
@pytest.mark.parametrize("m,n,kb", [(3, 300, 80), (100, 260, 80), (700, 2560, 40), (1100, 2050, 33)])
@pytest.mark.parametrize("off", [1, 2, 3])
def test_scales_at_any_address(fmt, grad, m, n, kb, off):
    """Scales are bytes: they may start anywhere."""
    k = kb * BLOCK[fmt]
    print_case(f"{'grad' if grad else 'matmul'} {fmt} m={m} n={n} k={k} scales + {off}")
    g = gen(m + off)
    xv, w = _x(g, 1, m, n if grad else k, torch.bfloat16), raw_weight(g, fmt, 1, n, k)
    s = w["scales"]
    buf = torch.full((s.numel() + 16,), 0x7F, device="cuda", dtype=torch.uint8)  # NVFP4's NaN around them
    shifted = buf[off:off + s.numel()].view(s.shape)
    shifted.copy_(s.view(torch.uint8))
    assert shifted.data_ptr() % 4 == off
    y = _call(grad)(xv, {**w, "scales": shifted}, fmt, out_dtype=torch.float32)
    check_product(y, xv, _wt(w, fmt, grad), 1)


def test_empty_products():
    fp = _m()
    g = gen(0)
    w = raw_weight(g, "nvfp4", 1, 32, 64)
    assert fp.fp4_matmul(torch.empty(1, 0, 64, device="cuda", dtype=torch.bfloat16), w, "nvfp4").shape == (1, 0, 32)
    none = raw_weight(g, "nvfp4", 1, 0, 64)
    assert fp.fp4_matmul(torch.empty(1, 5, 64, device="cuda"), none, "nvfp4").shape == (1, 5, 0)
    with pytest.raises(fp.Fp4Error):
        fp.fp4_matmul_grad(torch.empty(1, 5, 0, device="cuda"), none, "nvfp4")
