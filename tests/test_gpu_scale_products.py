"""Block-FP8 products whose two scales multiply to more or less than f32 holds, though the result
does not: the scales' product may neither become infinite (a zero sum then gives NaN) nor lose bits
as a subnormal.  Bars are those of the ordinary products: the product of the scales' mantissas and that
of the sum with it round by half a step each, as sx * sw and the fma do."""
import pytest

from gpu_util import gpu_ok, print_case, torch
from test_gpu_fp8_subnormal import _close
from test_gpu_matmul import _w64, _weight, _x64

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_ok(), reason="needs a GPU")]


def _m():
    import block_scaled_fp4_nvfp4_amd as m
    return m


# few rows in both forms, then every tile: 64 x 64 with and without the split of K, 128 x 128, 192 x 256, 256 x 256
SIZES = [(1, 1, 50, 512), (1, 4, 300, 384), (2, 16, 130, 1280), (1, 9, 64, 8192), (1, 40, 200, 128 * 26), (1, 512, 2560, 384),
         (1, 2100, 3001, 256), (1, 3801, 4001, 128), (1, 4101, 8200, 256)]


@pytest.mark.parametrize("b,m,n,k", SIZES)
@pytest.mark.parametrize("sx,sw", [(2.0 ** -82, 2.0 ** -60), (2.0 ** -30, 2.0 ** -106), (2.0 ** 70, 2.0 ** 62), (2.0 ** 24, 2.0 ** 106)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_products_beyond_f32(b, m, n, k, sx, sw, out):
    """Rows 0, 3, 6, .. have scales of about sx, the others ordinary ones, W of about sw: 1.0 to 2.2 times
    2^-142, 2^-136, 2^132 and 2^130 where they meet.  Where both are huge the codes are E4M3's smallest
    ones, so that y is finite, and one tile of W in two is ordinary.  The last block of row 0 is zero."""
    print_case(f"matmul scales b={b} m={m} n={n} k={k} {sx:.1e} {sw:.1e} {out}")
    g = torch.Generator(device="cuda")
    g.manual_seed(m + n)
    big = sx > 1
    w = _weight(g, b, n, k)
    codes = torch.randint(0, 4 if big else 0x7F, (b, m, k), device="cuda", generator=g).to(torch.uint8)
    codes |= torch.randint(0, 2, (b, m, k), device="cuda", generator=g).to(torch.uint8) << 7
    if big:
        w["codes"] = w["codes"] & 0x83
    codes[:, 0, k - 128:] = 0
    scales = torch.rand(b, m, k // 128, device="cuda", generator=g) + 0.5
    plain = {"codes": codes, "scales": scales.clone()}
    scales[:, ::3] *= sx
    w["scales"] = torch.rand(w["scales"].shape, device="cuda", generator=g) + 0.5
    w["scales"][..., slice((k // 128 - 1) % 2, None, 2) if big else slice(None)] *= sw
    q = {"codes": codes, "scales": scales}
    y = _m().fp8_matmul(q, w, out_dtype=out)
    assert bool(torch.isfinite(y).all())
    _close(y, _x64(q), _w64(w))
    # a row does not depend on the scales of its neighbours
    y2 = _m().fp8_matmul(plain, w, out_dtype=out)
    keep = [i for i in range(m) if i % 3]
    assert torch.equal(y[:, keep], y2[:, keep])


@pytest.mark.parametrize("m,n,k", [(600, 2000, 128 * 30), (20, 64, 128 * 97), (16, 64, 128 * 60), (2100, 3001, 128 * 26)])
@pytest.mark.parametrize("at", [0, -1])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_one_block_beyond_f32(m, n, k, at, out):
    """Only the first or the last of many blocks has such scales, in two rows and one tile of W; sums of
    zero times an infinite product of scales add nothing."""
    print_case(f"matmul scales of one block m={m} n={n} k={k} at={at} {out}")
    g = torch.Generator(device="cuda")
    g.manual_seed(m + k)
    w = _weight(g, 1, n, k)
    x = torch.randn(1, m, k, device="cuda", generator=g)
    q = _m().quantize(x, "fp8_row")
    at %= k // 128
    blk = slice(128 * at, 128 * at + 128)
    q["codes"][0, 1, blk] = 0
    q["codes"][0, m - 1, blk] = 1
    w["codes"][0, :128, blk] = 2
    ref = _m().fp8_matmul(q, w, out_dtype=out)
    q["scales"][0, 1, at] = 2.0 ** 90
    q["scales"][0, m - 1, at] = 2.0 ** -90
    w["scales"][0, 0, at] = 2.0 ** 60
    y = _m().fp8_matmul(q, w, out_dtype=out)
    assert bool(torch.isfinite(y).all())
    _close(y[:, :, :128], _x64(q), _w64(w)[:, :128])
    near = [i for i in range(m) if i not in (1, m - 1)]
    if n > 128:
        assert torch.equal(y[0, near, 128:], ref[0, near, 128:])


@pytest.mark.parametrize("m,n,k", [(40, 200, 128 * 26), (512, 2560, 384), (2100, 3001, 256), (4101, 8200, 256)])
@pytest.mark.parametrize("sx,sw", [(2.0 ** -99, 2.0 ** -23), (2.0 ** -101, 2.0 ** -25), (2.0 ** -98, 2.0 ** -30), (2.0 ** -61, 2.0 ** -62),
                                   (2.0 ** -64, 2.0 ** -64), (2.0 ** 119, 2.0 ** 6), (2.0 ** 120, 2.0 ** 8), (2.0 ** 61, 2.0 ** 61)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_scales_about_the_bounds_of_the_tables(m, n, k, sx, sw, out):
    """On either side of what the tile kernel takes in its ordinary form: [2^-100, 2^120] with [2^-24, 2^7],
    [2^-62, 2^62] with itself."""
    test_products_beyond_f32(1, m, n, k, sx, sw, out)


@pytest.mark.parametrize("m", [20, 300, 2100])
def test_padding_rows_of_anything(m):
    """Rows behind the last one in use that hold any bits: the others as without them."""
    print_case(f"matmul padding m={m}")
    g = torch.Generator(device="cuda")
    g.manual_seed(m)
    n, k = 2560, 512
    x = torch.randn(1, m, k, device="cuda", generator=g).to(torch.bfloat16)
    w = _weight(g, 1, n, k)
    x[:, m // 2:] = 0
    ref = _m().fp8_matmul(x, w)
    x[:, m // 2:] = torch.randint(-32768, 32768, (1, m - m // 2, k), device="cuda", generator=g, dtype=torch.int16).view(torch.bfloat16)
    assert torch.equal(_m().fp8_matmul(x, w)[:, :m // 2], ref[:, :m // 2])
