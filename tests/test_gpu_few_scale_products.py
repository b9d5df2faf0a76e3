"""The few-token layer with scales whose product is more or less than f32 holds, though what it makes of
them is not: the product may neither become infinite (a zero sum then gives NaN) nor lose bits as a
subnormal.  Bars are those of the layer's ordinary tests."""
import numpy as np
import pytest

from gpu_util import gpu_ok, host, print_case, rel_fro, torch
from test_gpu_few import _expected, _inputs, _layer

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_ok(), reason="needs a GPU")]


def _m():
    import block_scaled_fp4_nvfp4_amd as m
    return m


@pytest.mark.parametrize("T", [1, 6, 16])
def test_layer_with_gate_scales_below_f32(T):
    """x of 2^-70, gate scales 2^-52 of ordinary ones, up scales 2^120 of them: sx sw of the gate is
    about 2^-140, its sums and h are ordinary numbers."""
    print_case(f"few scales T={T}")
    layer = _layer("fp8", 7, 256, 128, 3, seed=T)
    layer.w13_scale[:, :1] *= 2.0 ** -52
    layer.w13_scale[:, 1:] *= 2.0 ** 120
    x, lg = _inputs(T, 7, 256, seed=T + 1)
    x = x * 2.0 ** -70
    y, ids, _ = _m().FewTokenLayer(layer, T)(x, lg)
    e_ids, _, e_y = _expected(layer, x, lg, None)
    np.testing.assert_array_equal(host(ids), e_ids)
    assert rel_fro(host(y) * 2.0 ** 70, e_y * 2.0 ** 70) <= 2e-3


def test_layer_with_zero_sums_of_huge_scales():
    """Gate and up blocks whose only non-zero codes meet zeros of x, with scales whose product with x's
    is infinite in f32: they add nothing."""
    print_case("few zero sums of huge scales")
    layer = _layer("fp8", 5, 256, 128, 2, seed=1)
    x, lg = _inputs(4, 5, 256, seed=2)
    x = x * 2.0 ** 40
    layer.w13_scale *= 2.0 ** -40
    x[:, 128] = 0.0
    layer.w13[:, :, 128:] = 0
    ref = [t.clone() for t in _m().FewTokenLayer(layer, 4)(x, lg)]
    layer.w13[:, :, 128] = 0x7E
    layer.w13_scale[:, :, 1] = 2.0 ** 100
    for a, b in zip(ref, _m().FewTokenLayer(layer, 4)(x, lg)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [2, 9])
def test_nvfp4_layer_with_tiny_tensor_scales(T):
    """NVFP4 / NVFP4 with w2's and h's tensor scales about 2^-75 each: their product, with the routing
    weight, is a subnormal f32 of few bits, y is not (its block scales and codes bring 2^22)."""
    print_case(f"few tensor scales T={T}")
    layer = _layer("nvnv", 6, 256, 128, 2, seed=T)
    x, lg = _inputs(T, 6, 256, seed=T)
    for name, f in (("w13_scale_2", 2.0 ** -31), ("w2_scale_2", 2.0 ** -58)):
        setattr(layer, name, getattr(layer, name) * f)
    y, ids, _ = _m().FewTokenLayer(layer, T)(x, lg)
    e_ids, _, e_y = _expected(layer, x, lg, None)
    np.testing.assert_array_equal(host(ids), e_ids)
    assert rel_fro(host(y).astype(np.float64) * 2.0 ** 100, e_y * 2.0 ** 100) <= 2e-3
