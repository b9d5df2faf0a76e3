"""Results of fp4_matmul and fp4_matmul_grad next to f32's largest value, whatever the NVFP4 tensor scale: sums of
positive products, so that no partial sum is larger than the result, which is finite."""
import pytest

from gpu_util import gpu_ok, print_case, torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_ok(), reason="needs a GPU")]

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
LARGE = 3.2e38  # f32 ends at 3.4028e38, bf16 at 3.3895e38


# few rows in one, two and four blocks, tiles, shared tiles that are joined; odd sizes
@pytest.mark.parametrize("b,m,n,k", [(1, 1, 48, 64), (2, 30, 35, 80), (1, 60, 48, 320), (2, 100, 130, 96), (1, 16, 640, 9600), (1, 70, 64, 9600),
                                     (2, 300, 1001, 272)])
@pytest.mark.parametrize("S", [1.0, 1.75, 0.375, 40.0])
@pytest.mark.parametrize("grad", [False, True], ids=["product", "gradient"])
@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_large_results_are_finite(b, m, n, k, S, grad, x):
    """All weights 6 x 448 S, all x alike: result c 2688 S x.  Exact operands, so that only the sums round: c additions (three
    terms each of f32 x) of half a step 2^-24 and the tensor scale's factor; bf16 results half a step 2^-8 more."""
    import block_scaled_fp4_nvfp4_amd as fp
    print_case(f"large results b={b} m={m} n={n} k={k} S={S} grad={grad} {x}")
    c = n if grad else k
    scales = torch.tensor([S] + [1.25 * S] * (b - 1), device="cuda")
    w = {"codes": torch.full((b, n, k // 2), 0x77, dtype=torch.uint8, device="cuda"),
         "scales": torch.full((b, n, k // 16), 0x7E, dtype=torch.uint8, device="cuda"), "tensor_scale": scales}
    one = (LARGE / (c * 2688 * scales.double())).to(DT[x])
    xv = one.reshape(b, 1, 1).expand(b, m, c).contiguous()
    want = (c * 2688 * scales.double() * one.double()).reshape(b, 1, 1)
    assert float(want.max()) < 1.01 * LARGE
    for out in ("f32", "bf16"):
        for sign in (1, -1):
            y = (fp.fp4_matmul_grad if grad else fp.fp4_matmul)(sign * xv, w, "nvfp4", out_dtype=DT[out])
            tol = ((3 if x == "f32" else 1) * c + 2) * 2.0 ** -24 + (2.0 ** -8 if out == "bf16" else 0.0)
            assert bool((((sign * y.double() - want) / want).abs() <= tol).all()), float(y.double().abs().max())
