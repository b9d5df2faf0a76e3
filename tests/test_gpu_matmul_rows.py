"""A row of y depends on its own row of x alone: with every other row replaced (ordinary values, zeros,
the largest finite ones, infinities and NaN) it keeps its bits, in each kernel's range of rows and for
x as codes, bf16 and f32; a matrix of a batch likewise."""
import pytest

from gpu_util import gpu_ok, print_case, torch
from test_gpu_matmul import _case

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_ok(), reason="needs a GPU")]


def _m():
    import block_scaled_fp4_nvfp4_amd as m
    return m


# few rows in their three forms, then tiles of 64 x 64 (K split and not), 128 x 128, 256 x 256 and 192 x 256
SIZES = [(2, 100, 512), (4, 100, 512), (5, 100, 1280), (16, 130, 8192), (17, 64, 2560), (40, 200, 128 * 26), (512, 2560, 384),
         (2100, 3001, 256), (3801, 4001, 128), (4101, 8200, 256)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_other_rows_do_not_matter(m, n, k, out):
    print_case(f"matmul rows m={m} n={n} k={k} {out}")
    rows = sorted({1, m - 1, m // 2})
    for dtype in (torch.bfloat16, torch.float32):
        x, w = _case(m + n, 1, m, n, k, dtype)
        q = _m().quantize(x, "fp8_row")
        ref = [t[:, rows].clone() for t in (_m().fp8_matmul(x, w, out_dtype=out), _m().fp8_matmul(q, w, out_dtype=out))]
        for fill in (0.0, float(torch.finfo(dtype).max), float("inf"), float("nan"), None):
            x2 = torch.full_like(x, fill) if fill is not None else _case(m + n + 1, 1, m, n, k, dtype)[0]
            x2[:, rows] = x[:, rows]
            q2 = {key: torch.full_like(q[key], 0x7F if key == "codes" else fill if fill is not None else 3.0) for key in ("codes", "scales")}
            for key in q2:
                q2[key][:, rows] = q[key][:, rows]
            got = [_m().fp8_matmul(x2, w, out_dtype=out), _m().fp8_matmul(q2, w, out_dtype=out)]
            assert all(torch.equal(a, b[:, rows]) for a, b in zip(ref, got)), (dtype, fill)


@pytest.mark.parametrize("m", [3, 16, 70])
def test_other_matrices_do_not_matter(m):
    print_case(f"matmul matrices m={m}")
    x, w = _case(m, 3, m, 300, 384)
    y = _m().fp8_matmul(x, w)
    x2, w2 = _case(m + 1, 3, m, 300, 384)
    x2[0], x2[2] = float("nan"), 0.0
    x2[1] = x[1]
    for key in ("codes", "scales"):
        w2[key][1] = w[key][1]
    w2["scales"][0] = float("inf")
    assert torch.equal(y[1], _m().fp8_matmul(x2, w2)[1])


@pytest.mark.parametrize("m", [1, 4, 16, 17, 300])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_not_finite_shows_in_its_row(m, bad):
    """Outside of what the operator asks of x, but never a finite result: the block's codes are NaN."""
    print_case(f"matmul not finite m={m} {bad}")
    for dtype in (torch.bfloat16, torch.float32):
        x, w = _case(m, 1, m, 100, 384, dtype)
        y = _m().fp8_matmul(x, w)
        x[0, m - 1, 200] = bad
        y2 = _m().fp8_matmul(x, w)
        assert bool(torch.isnan(y2[0, m - 1]).all()) and torch.equal(y[:, :m - 1], y2[:, :m - 1])
