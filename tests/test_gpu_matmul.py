"""fp8_block_matmul against a float64 product of the exact values of its codes.

Tolerances, from the number formats: with P = sum_k |x_k w_k| of an output's
dequantized operands,
  bf16 results  half a bf16 step of the result (2^-8 relative) and 2^-14 P for
                the E4M3 MFMA, which keeps 16 or more bits of a block's sum below
                its largest partial sum (at most P), and the f32 scaling;
  f32 results   (128 + K / 128 + 4) 2^-23 P: at most 128 additions in a block,
                one per block and the scalings, each off by a step of its
                partial sum at most; and 1e-6 in the Frobenius norm.
"""
import numpy as np
import pytest

from oracle import quant

from gpu_util import gpu_ok, host, print_case, rel_fro, torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_ok(), reason="needs a GPU")]


def _m():
    import block_scaled_fp4_nvfp4_amd as m
    return m


def _weight(g, b, n, k):
    """W ~ N(0, 0.02) quantized by the library on rows padded to 128; the first n rows' codes."""
    pad = (n + 127) // 128 * 128
    w = torch.zeros(b, pad, k, device="cuda")
    w[:, :n] = torch.randn(b, n, k, device="cuda", generator=g) * 0.02
    q = _m().quantize(w, "fp8_block")
    return {"codes": q["codes"][:, :n].contiguous(), "scales": q["scales"]}


def _case(seed, b, m, n, k, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = (torch.randn(b, m, k, device="cuda", generator=g) * torch.exp(torch.randn(b, m, 1, device="cuda", generator=g)))
    return x.to(dtype), _weight(g, b, n, k)


def _w64(w):
    codes, scales = w["codes"], w["scales"]
    v = codes.view(torch.float8_e4m3fn).double()
    s = scales.double().repeat_interleave(128, -2)[..., :codes.shape[-2], :].repeat_interleave(128, -1)
    return v * s


def _x64(q):
    return q["codes"].view(torch.float8_e4m3fn).double() * q["scales"].double().repeat_interleave(128, -1)


def _check(y, xd, wd):
    """y against the float64 product of xd [B, M, K] and wd [B, N, K]."""
    e = torch.matmul(xd, wd.transpose(-1, -2).contiguous())
    p = torch.matmul(xd.abs(), wd.abs().transpose(-1, -2).contiguous())
    k = xd.shape[-1]
    err = (y.double() - e).abs()
    if y.dtype == torch.bfloat16:
        tol = 2.0 ** -8 * e.abs() + 2.0 ** -14 * p
    else:
        tol = (128 + k / 128 + 4) * 2.0 ** -23 * p
        assert rel_fro(host(y), host(e)) <= 1e-6
    bad = err > tol
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} outside, worst {float((err / tol.clamp(min=1e-300)).max()):.3g} of the tolerance"


SIZES = [(1, 1, 1, 128), (1, 1, 16, 256), (1, 2, 17, 128), (1, 15, 130, 384), (1, 16, 128, 2560), (1, 17, 257, 640),
         (1, 33, 64, 1280), (1, 63, 1000, 256), (1, 64, 127, 512), (1, 65, 640, 128), (1, 100, 129, 1152), (3, 7, 48, 128),
         (2, 129, 300, 256), (1, 255, 513, 384), (1, 256, 256, 1024), (1, 300, 2560, 640), (5, 70, 512, 128),
         (1, 513, 1290, 2560), (1, 1, 4099, 10240), (1, 9, 250, 10368), (1, 700, 40, 5120)]


@pytest.mark.parametrize("b,m,n,k", SIZES)
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_codes_and_values(b, m, n, k, out):
    print_case(f"matmul b={b} m={m} n={n} k={k} {out}")
    x, w = _case(b * 7 + m * 3 + n + k, b, m, n, k)
    q = _m().quantize(x, "fp8_row")
    y = _m().fp8_matmul(q, w, out_dtype=out)
    assert y.shape == (b, m, n) and y.dtype == out
    _check(y, _x64(q), _w64(w))
    # quantization within the call: the same codes, hence the same bits
    y2 = _m().fp8_matmul(x, w, out_dtype=out)
    assert torch.equal(y, y2)


@pytest.mark.parametrize("m", [1, 5, 40, 200])
def test_f32_values_and_oracle_quantization(m):
    """f32 x through the oracle's quantizer of rows (independent of the library's)."""
    print_case(f"matmul f32 x m={m}")
    n, k = 200, 512
    x, w = _case(m, 1, m, n, k, torch.float32)
    o = quant.quantize_fp8_rows(host(x[0]).astype(np.float64))
    xd = torch.from_numpy(np.asarray(quant.dequantize_fp8_rows(o["codes"], o["scales"]))).cuda()[None]
    for out in (torch.bfloat16, torch.float32):
        _check(_m().fp8_matmul(x, w, out_dtype=out), xd, _w64(w))


@pytest.mark.parametrize("m", [3, 20, 150])
def test_zero_blocks_extremes_and_rounding_borders(m):
    """Zero rows and zero 128-blocks (scale 0), values at the E4M3 rounding borders, very large and
    very small rows; a row's neighbours do not change it."""
    print_case(f"matmul borders m={m}")
    g = torch.Generator(device="cuda")
    g.manual_seed(m)
    k, n = 512, 144
    w = _weight(g, 1, n, k)
    grid = torch.tensor([1.0625, 1.1875, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, 447.0, 448.0, 432.0, 1.0], device="cuda")
    x = grid[torch.randint(0, 10, (1, m, k), device="cuda", generator=g)] * (torch.randint(0, 2, (1, m, k), device="cuda", generator=g) * 2 - 1)
    x[..., ::128] = 448.0   # sigma = 1: the grid's values are the quotients
    x[:, 0] = 0
    x[:, :, 128:256] = 0
    x[:, 1] *= 2.0 ** 80
    x[:, 2] *= 2.0 ** -80
    for dt in (torch.bfloat16, torch.float32):
        xx = x.to(dt)
        q = _m().quantize(xx, "fp8_row")
        o = quant.quantize_fp8_rows(host(xx[0].float()).astype(np.float64))
        np.testing.assert_array_equal(host(q["codes"][0]) & 0x7F, np.asarray(o["codes"]) & 0x7F)
        for out in (torch.bfloat16, torch.float32):
            y = _m().fp8_matmul(xx, w, out_dtype=out)
            assert torch.equal(y, _m().fp8_matmul(q, w, out_dtype=out))
            assert float(y[0, 0].abs().max()) == 0.0
            _check(y, _x64(q), _w64(w))
            assert torch.equal(_m().fp8_matmul(xx[:, 1:2], w, out_dtype=out)[0, 0], _m().fp8_matmul(xx[:, 1:2].clone(), w, out_dtype=out)[0, 0])


@pytest.mark.parametrize("b,m,n,k", [(1, 5, 37, 256), (1, 70, 129, 384), (2, 130, 263, 256), (1, 17, 16, 128)])
def test_nothing_outside_y_is_written(b, m, n, k):
    print_case(f"matmul canary b={b} m={m} n={n} k={k}")
    x, w = _case(5, b, m, n, k)
    for out in (torch.bfloat16, torch.float32):
        buf = torch.full((b * m * n + 2 * 4096,), -7.0, dtype=out, device="cuda")
        y = buf[4096:4096 + b * m * n].view(b, m, n)
        need = _m().fp8_matmul_workspace_size(x.dtype, b, m, n, k)
        ws = torch.full((need + 4096,), 171, dtype=torch.uint8, device="cuda")
        got = _m().fp8_matmul(x, w, out_dtype=out, out=y, workspace=ws[:need])
        assert got.data_ptr() == y.data_ptr()
        assert bool((buf[:4096] == -7).all()) and bool((buf[4096 + b * m * n:] == -7).all())
        assert bool((ws[need:] == 171).all())
        assert torch.equal(y, _m().fp8_matmul(x, w, out_dtype=out))


def test_two_dimensional_and_empty():
    x, w = _case(9, 1, 6, 50, 128)
    w2 = {"codes": w["codes"][0], "scales": w["scales"][0]}
    y = _m().fp8_matmul(x[0], w2)
    assert y.shape == (6, 50) and torch.equal(y, _m().fp8_matmul(x, w)[0])
    assert _m().fp8_matmul(x[0, :0], w2).shape == (0, 50)


def test_streams_and_captured_graphs():
    """On a side stream; two graphs with a workspace each, replayed in turns with new inputs and eager
    work between, every replay equal to the eager product of the same inputs."""
    print_case("matmul streams and graphs")
    cases = [_case(21, 1, 12, 300, 512), _case(22, 1, 90, 260, 256)]
    eager = [_m().fp8_matmul(x, w) for x, w in cases]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        side = [_m().fp8_matmul(x, w) for x, w in cases]
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(eager, side):
        assert torch.equal(a, b)
    graphs, outs = [], []
    for x, w in cases:
        ws = torch.empty(max(1, _m().fp8_matmul_workspace_size(x.dtype, *x.shape[:2], w["codes"].shape[1], x.shape[2])),
                         dtype=torch.uint8, device="cuda")
        y = torch.empty(1, x.shape[1], w["codes"].shape[1], dtype=torch.bfloat16, device="cuda")
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            _m().fp8_matmul(x, w, out=y, workspace=ws)
        graphs.append(gr)
        outs.append(y)
    for rep in range(4):
        for (x, w), gr, y in zip(cases, graphs, outs):
            x.copy_(torch.roll(x, 1, dims=1) * 1.5)
            gr.replay()
            assert torch.equal(y, _m().fp8_matmul(x, w)), rep
        torch.cuda.synchronize()


@pytest.mark.parametrize("b,m,n,k", [(1, 2100, 3001, 640), (1, 4101, 4103, 256), (2, 1901, 4007, 256), (1, 3801, 4001, 128)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_large_products_with_ragged_edges(b, m, n, k, out):
    """Sizes at which the larger tiles are chosen; neither m nor n is a multiple of one."""
    print_case(f"matmul large b={b} m={m} n={n} k={k} {out}")
    x, w = _case(b + m + n + k, b, m, n, k)
    q = _m().quantize(x, "fp8_row")
    y = _m().fp8_matmul(q, w, out_dtype=out)
    _check(y, _x64(q), _w64(w))
    assert torch.equal(y, _m().fp8_matmul(x, w, out_dtype=out))


@pytest.mark.parametrize("b,m,n,k", [(1, 40, 200, 128 * 17), (1, 70, 129, 128 * 54), (2, 100, 130, 8192), (1, 20, 64, 128 * 97)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_few_tiles_of_many_steps(b, m, n, k, out):
    """Sizes whose K is split between waves: runs of unequal length, more steps than a table of scales holds."""
    print_case(f"matmul long b={b} m={m} n={n} k={k} {out}")
    x, w = _case(b + m + n + k, b, m, n, k)
    q = _m().quantize(x, "fp8_row")
    y = _m().fp8_matmul(q, w, out_dtype=out)
    _check(y, _x64(q), _w64(w))
    assert torch.equal(y, _m().fp8_matmul(x, w, out_dtype=out))
    assert torch.equal(y, _m().fp8_matmul(q, w, out_dtype=out))
