"""The few-token layer at 512 experts of hidden 2560, intermediate 640, top 10, against the same layer
through moe_fp4_route and moe_fp4_forward (other kernels): ids equal, y within the sum of both bars
(1e-5 each with plain activations, 2e-3 each with quantized ones)."""
import pytest

from gpu_util import gpu_ok, host, print_case, rel_fro, torch
from test_gpu_few import MODES, _gen, _inputs, _layer

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_ok(), reason="needs a GPU")]


@pytest.mark.parametrize("mode", MODES)
def test_full_size(mode):
    import block_scaled_fp4_nvfp4_amd as m
    plain = MODES[mode][1] == "none"
    layer = _layer(mode, 512, 2560, 640, 10, seed=1, shared=0 if plain else 1280)
    few = m.FewTokenLayer(layer, 16)
    for T in (1, 2, 7, 16):
        print_case(f"few full size {mode} T={T}")
        x, lg = _inputs(T, 512, 2560, seed=T)
        bias = torch.randn(512, device="cuda", generator=_gen(T)) if T % 2 else None
        y, ids, w = few(x, lg, bias)
        r_ids, r_w = m.route(lg, 10, bias)
        assert torch.equal(ids, r_ids) and torch.allclose(w, r_w, rtol=2.0 ** -22, atol=0)
        assert rel_fro(host(y), host(m.moe_forward(layer, x, r_ids, r_w))) <= (2e-5 if plain else 4e-3)
        assert all(torch.equal(a, b) for a, b in zip((y, ids, w), few(x, lg, bias)))
    del layer, few
    torch.cuda.empty_cache()
