"""FP8 rows whose 128-blocks are so small that their scale is a subnormal f32 of a few units: the
scale rounds far below amax / 448, the quotients pass E4M3's largest value and must saturate there,
as fp4_quantize and the oracle do."""
import numpy as np
import pytest

from oracle import quant

from gpu_util import gpu_ok, host, print_case, torch
from test_gpu_few import _layer
from test_gpu_matmul import _w64, _weight, _x64

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_ok(), reason="needs a GPU")]


def _m():
    import block_scaled_fp4_nvfp4_amd as m
    return m


def _close(y, xd, wd):
    """y against the float64 product of xd [B, M, K] and wd [B, N, K], with P the sum of the products'
    magnitudes.  bf16: half a step of the result (2^-8), and the E4M3 MFMA adds the products in eights,
    each aligned to the eight's largest and cut 14 bits below its leading bit: seven cuts of less than
    2^-14 of a product that P holds.  Both: f32 additions (128 in a block at most, one per block) and
    scalings, half a step (2^-24) each, of at most P.  A step is 2^-133 (bf16) or 2^-149 (f32) at least:
    half of it for the result and for each block's scaled sum."""
    e = torch.matmul(xd, wd.transpose(-1, -2).contiguous())
    p = torch.matmul(xd.abs(), wd.abs().transpose(-1, -2).contiguous())
    tol = (128 + xd.shape[-1] / 128 + 4) * 2.0 ** -24 * p + xd.shape[-1] / 128 * 2.0 ** -150
    if y.dtype == torch.bfloat16:
        tol = 2.0 ** -8 * e.abs() + (7 * 2.0 ** -14 * p + tol) * (1 + 2.0 ** -8) + 2.0 ** -134
    err = (y.double() - e).abs()
    assert bool((err <= tol).all()), f"worst {float((err / tol.clamp(min=1e-300)).max()):.3g} of the tolerance"


def _tiny_rows(m, k, seed, lo, hi):
    """f32 [1, m, k]: every 128-block's largest magnitude is n units of 2^-149, n spread over lo .. hi."""
    r = np.random.default_rng(seed)
    n = np.linspace(lo, hi, m * (k // 128)).round().astype(np.int64).reshape(m, k // 128, 1)
    v = r.integers(-n, n + 1, (m, k // 128, 128))
    v[..., 17] = n[..., 0] * r.choice([-1, 1], (m, k // 128))
    bits = (np.abs(v).astype(np.uint32) | np.where(v < 0, np.uint32(1 << 31), np.uint32(0))).reshape(1, m, k)
    return torch.from_numpy(bits.view(np.float32)).cuda()


@pytest.mark.parametrize("m", [1, 3, 4, 16, 17, 90, 300])
@pytest.mark.parametrize("lo,hi", [(1, 400), (200, 6500), (6500, 1 << 20)])
def test_rows_of_a_few_units(m, lo, hi):
    print_case(f"matmul subnormal rows m={m} {lo}..{hi}")
    g = torch.Generator(device="cuda")
    g.manual_seed(m)
    k, n = 384, 80
    w = _weight(g, 1, n, k)
    w["scales"] *= 2.0 ** 100  # y in f32's normal range
    x = _tiny_rows(m, k, m + lo, lo, hi)
    q = _m().quantize(x, "fp8_row")
    o = quant.quantize_fp8_rows(host(x[0]).astype(np.float64))
    np.testing.assert_array_equal(host(q["scales"][0]), o["scales"])
    np.testing.assert_array_equal(host(q["codes"][0]) & 0x7F, np.asarray(o["codes"]) & 0x7F)
    for out in (torch.bfloat16, torch.float32):
        y = _m().fp8_matmul(x, w, out_dtype=out)
        assert torch.equal(y, _m().fp8_matmul(q, w, out_dtype=out))
        _close(y, _x64(q), _w64(w))


@pytest.mark.parametrize("most", [3, 10, 16])
@pytest.mark.parametrize("T", [1, 5, 16])
def test_h_of_a_few_units(most, T):
    """The block-FP8 layer with h = 196 k units of 2^-149, k up to `most` (588 and 1960 units: quotients
    of 588 and 490), exactly: one non-zero x of code 448 and scale 1, gate 28 (SiLU(28) = 28 in f32) and
    up rows of 7 k units.  h meets the MFMA as bf16 terms, whose step is 2^-133 at this size: y is
    within that step, times the magnitudes of W2, of the definition."""
    print_case(f"few subnormal h most={most} T={T}")
    E, H, I, k = 3, 128, 128, 2
    layer = _layer("fp8", E, H, I, k, seed=most)
    one = int(torch.tensor(1.0).to(torch.float8_e4m3fn).view(torch.uint8))
    layer.w13.zero_()
    layer.w13[:, :I, 5] = one
    ks = torch.arange(I) % (most + 1)
    layer.w13[:, I:, 5] = (ks / 64).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    layer.w13_scale[:, 0] = 2.0 ** -4
    layer.w13_scale[:, 1] = torch.tensor([1], dtype=torch.int32, device="cuda").view(torch.float32)  # 2^-149
    x = torch.zeros(T, H, device="cuda", dtype=torch.bfloat16)
    x[:, 5] = 448.0
    lg = torch.randn(T, E, device="cuda", generator=torch.Generator(device="cuda").manual_seed(T))
    y, ids, w = _m().FewTokenLayer(layer, T)(x, lg)
    h = (196 * ks).double().numpy() * 2.0 ** -149
    o = quant.quantize_fp8_rows(h[None])
    hq = quant.dequantize_fp8_rows(o["codes"], o["scales"])[0]
    w2 = host(_w64({"codes": layer.w2, "scales": layer.w2_scale}))
    ids, w = host(ids), host(w).astype(np.float64)
    for t in range(T):
        e = sum(w[t, j] * (w2[ids[t, j]] @ hq) for j in range(k))
        tol = 2.0 ** -133 * sum(w[t, j] * np.abs(w2[ids[t, j]]).sum(1) for j in range(k)) + 2.0 ** -148
        got = host(y[t]).astype(np.float64)
        assert np.isfinite(got).all() and (np.abs(got - e) <= tol).all(), t
