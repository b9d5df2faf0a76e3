"""A decode step as a user writes it: a block-FP8 dense layer, the routed-expert
layer on its output and another dense layer on that one's, with a residual, for
1, 5 and 16 tokens; eager and as a captured graph.  Every stage is checked
against float64 on the inputs it was given, with its own test's bar."""
import numpy as np
import pytest

from gpu_util import gpu_ok, host, print_case, rel_fro, torch
from test_gpu_few import _expected, _gen, _layer
from test_gpu_matmul import _check, _w64, _weight, _x64

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_ok(), reason="needs a GPU")]


def _m():
    import block_scaled_fp4_nvfp4_amd as m
    return m


@pytest.mark.parametrize("mode", ["nv", "nvnv", "mx", "mxmx", "fp8"])
@pytest.mark.parametrize("T", [1, 5, 16])
def test_decode_step(mode, T):
    print_case(f"decode step {mode} T={T}")
    m, g = _m(), _gen(T)
    H, E, k = 512, 24, 4
    layer = _layer(mode, E, H, 256, k, seed=T, shared=128)
    few = m.FewTokenLayer(layer, 16)
    w_in, w_gate, w_out = (_weight(g, 1, n, H) for n in (H, E, 2 * H))
    x = torch.randn(1, T, H, device="cuda", generator=g).to(torch.bfloat16)

    def step(x):
        a = m.fp8_matmul(x, w_in)
        logits = m.fp8_matmul(a, w_gate, out_dtype=torch.float32)
        y, ids, w = few(a[0], logits[0])
        r = (y[None] + a.float())
        return a, logits, y, ids, w, r, m.fp8_matmul(r, w_out)

    out = step(x)
    a, logits, y, ids, w, r, z = out
    _check(a, _x64(m.quantize(x, "fp8_row")), _w64(w_in))
    _check(logits, _x64(m.quantize(a, "fp8_row")), _w64(w_gate))
    e_ids, e_w, e_y = _expected(layer, a[0], logits[0], None)
    np.testing.assert_array_equal(host(ids), e_ids)
    np.testing.assert_array_max_ulp(host(w), e_w, maxulp=1)
    assert rel_fro(host(y), e_y) <= 2e-3
    _check(z, _x64(m.quantize(r, "fp8_row")), _w64(w_out))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = step(x)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(out, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step(x)
    for rep in range(3):
        x.copy_(torch.roll(x, 1 + rep, dims=2) * 0.75)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in kept]
        assert all(torch.equal(p, q) for p, q in zip(got, step(x))), rep
