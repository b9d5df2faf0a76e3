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


def test_two_calls_at_once():
    """Both operators on two streams at the same time, a workspace each: every result as if alone."""
    print_case("two streams at once")
    m, g = _m(), _gen(3)
    H, E, k = 512, 40, 4
    layer = _layer("nv", E, H, 256, k, seed=2)
    w = _weight(g, 1, 1024, H)
    xs = [torch.randn(1, t, H, device="cuda", generator=g).to(torch.bfloat16) for t in (3, 16)]
    lg = [torch.randn(t, E, device="cuda", generator=g) for t in (3, 16)]
    few = [m.FewTokenLayer(layer, 16) for _ in xs]
    wide = [torch.randn(1, 40 + 60 * i, H, device="cuda", generator=g).to(torch.bfloat16) for i in range(2)]
    alone = [(*f(x[0], l), m.fp8_matmul(a, w)) for f, x, l, a in zip(few, xs, lg, wide)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[] for _ in xs]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append((*few[i](xs[i][0], lg[i]), m.fp8_matmul(wide[i], w)))
    torch.cuda.synchronize()
    for i, ref in enumerate(alone):
        for r in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(ref, r))


@pytest.mark.parametrize("mode", ["nv", "nvnv", "mx", "mxmx", "fp8"])
def test_what_a_workspace_held_does_not_matter(mode):
    """Workspaces full of NaN bytes, tokens with some, one and no experts selected."""
    print_case(f"poisoned workspace {mode}")
    m, g = _m(), _gen(4)
    layer = _layer(mode, 12, 256, 128, 3, seed=5, shared=128)
    x = torch.randn(6, 256, device="cuda", generator=g).to(torch.bfloat16)
    lg = torch.randn(6, 12, device="cuda", generator=g)
    lg[1] = lg[5] = float("-inf")
    lg[2, 1:] = float("-inf")
    few = m.FewTokenLayer(layer, 6)
    ref = [t.clone() for t in few(x, lg)]
    for fill in (255, 0, 127):
        few.workspace.fill_(fill)
        assert all(torch.equal(a, b) for a, b in zip(ref, few(x, lg))), fill
    w = _weight(g, 1, 200, 256)
    xb = torch.randn(1, 50, 256, device="cuda", generator=g).to(torch.bfloat16)
    ws = torch.empty(m.fp8_matmul_workspace_size(xb.dtype, 1, 50, 200, 256), dtype=torch.uint8, device="cuda")
    y = m.fp8_matmul(xb, w)
    for fill in (255, 0):
        ws.fill_(fill)
        assert torch.equal(y, m.fp8_matmul(xb, w, workspace=ws)), fill
