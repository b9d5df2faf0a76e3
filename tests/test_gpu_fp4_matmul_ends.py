"""fp4_matmul and fp4_matmul_grad at the longest sums and rows that they take: 2^22 products, k = 2^26."""
import pytest

from gpu_util import gpu_ok, print_case, torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_ok(), reason="needs a GPU")]

from head_util import check_product, gen, raw_weight, w64  # noqa: E402


@pytest.mark.parametrize("fmt,m,x", [("nvfp4", 1, "bf16"), ("mxfp4", 70, "bf16"), ("nvfp4", 20, "f32")])
def test_longest_sums(fmt, m, x):
    import block_scaled_fp4_nvfp4_amd as fp
    n, k = 21, 1 << 22
    print_case(f"matmul {fmt} m={m} n={n} k={k} {x}")
    g = gen(m)
    xv, w = torch.randn(1, m, k, device="cuda", generator=g).to(torch.bfloat16 if x == "bf16" else torch.float32), raw_weight(g, fmt, 1, n, k)
    y = fp.fp4_matmul(xv, w, fmt, out_dtype=torch.float32)
    check_product(y, xv, w64(w, fmt).transpose(-1, -2), 3 if x == "f32" else 1)


@pytest.mark.parametrize("fmt,n", [("nvfp4", 40), ("mxfp4", 70)])
def test_longest_rows_of_a_gradient(fmt, n):
    """The first and the last columns; a canary behind."""
    import block_scaled_fp4_nvfp4_amd as fp
    m, k, B = 2, 1 << 26, 16 if fmt == "nvfp4" else 32
    print_case(f"grad {fmt} m={m} n={n} k={k}")
    g = gen(n)
    dy, w = torch.randn(1, m, n, device="cuda", generator=g).bfloat16(), raw_weight(g, fmt, 1, n, k)
    res = torch.full((m * k + 4096,), 7.0, device="cuda")
    out = res[:m * k].view(1, m, k)
    fp.fp4_matmul_grad(dy, w, fmt, out_dtype=torch.float32, out=out)
    assert bool((res[m * k:] == 7.0).all())
    for at in (0, k // 2 - 512, k - 1024):
        part = {**w, "codes": w["codes"][..., at // 2:at // 2 + 512], "scales": w["scales"][..., at // B:(at + 1024) // B]}
        check_product(out[..., at:at + 1024], dy, w64(part, fmt), 1)


@pytest.mark.parametrize("m", [1, 33])
def test_longest_sums_of_a_gradient(m):
    import block_scaled_fp4_nvfp4_amd as fp
    n, k = 1 << 22, 48
    print_case(f"grad nvfp4 m={m} n={n} k={k}")
    g = gen(m)
    dy, w = torch.randn(1, m, n, device="cuda", generator=g).bfloat16(), raw_weight(g, "nvfp4", 1, n, k)
    check_product(fp.fp4_matmul_grad(dy, w, "nvfp4", out_dtype=torch.float32), dy, w64(w, "nvfp4"), 1)
