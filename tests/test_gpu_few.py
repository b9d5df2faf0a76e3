"""moe_fp4_forward_few (a whole routed-expert layer for 1 to 16 tokens, from
router logits to y) against a float64 evaluation with the oracle's routing
rule, dequantization and activation quantizers.

Bars: ids exact, weights within one f32 ulp (both are f64 softmaxes rounded
once; their exp and sum differ in the last bits); y in f32 within 1e-5 in the
Frobenius norm where activations are not quantized (f32 sums of up to 4096
products and the f32 SiLU; the bar of the layer's own tests), 2e-3 where they
are (an intermediate value within f32 error of a rounding border may round
the other way, which moves y by one code's step of one of its inputs); y in
bf16 equal to the f32 y rounded once."""
import numpy as np
import pytest

from oracle import moe

from gpu_util import dev, gpu_ok, host, print_case, rel_fro, torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_ok(), reason="needs a GPU")]

MODES = {"nv": ("nvfp4", "none"), "mx": ("mxfp4", "none"), "nvnv": ("nvfp4", "nvfp4"), "mxmx": ("mxfp4", "mxfp8"),
         "fp8": ("fp8_block", "fp8_row")}


def _m():
    import block_scaled_fp4_nvfp4_amd as m
    return m


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _layer(mode, E, H, I, k, seed, shared=0):
    m, g = _m(), _gen(seed)
    w_fmt, a_fmt = MODES[mode]
    draw = lambda *s: (torch.randn(*s, device="cuda", generator=g) * 0.05).to(torch.bfloat16)
    q13, q2 = m.quantize(draw(E, 2 * I, H), w_fmt), m.quantize(draw(E, H, I), w_fmt)
    layer = m.MoELayer(w_fmt, a_fmt, E, H, I, k, q13["codes"], q13["scales"], q2["codes"], q2["scales"],
                       q13["tensor_scale"], q2["tensor_scale"])
    if shared:
        a, b = m.quantize(draw(2 * shared, H), "mxfp8"), m.quantize(draw(H, shared), "mxfp8")
        layer.shared_inter = shared
        layer.ws13, layer.ws13_scale, layer.ws2, layer.ws2_scale = a["codes"], a["scales"], b["codes"], b["scales"]
        layer.shared_gate = draw(H)
    return layer


def _deq(codes, scales, ts, fmt):
    q = {"codes": host(codes), "scales": host(scales)}
    if ts is not None:
        q["tensor_scale"] = np.float32(float(ts))
    if fmt in ("nvfp4", "mxfp4"):
        q = moe.unpacked(q)
    return moe.dequantize_weight(q, fmt)


def _expected(layer, x, logits, bias):
    """ids, weights, y in float64 (numpy)."""
    lp = host(logits).astype(np.float32)
    if bias is not None:
        lp = (lp + host(bias)[None, :]).astype(np.float32)
    T, E = lp.shape
    k, I = layer.top_k, layer.inter
    ids, wts = np.full((T, k), -1, np.int32), np.zeros((T, k), np.float32)
    for t in range(T):
        ok = [e for e in range(E) if lp[t, e] > -np.inf]
        if not ok:
            continue
        sel = sorted(ok, key=lambda e: (-float(lp[t, e]), e))[:k]
        o_ids, o_w = moe.route(lp[t:t + 1, sel], None, len(sel))
        np.testing.assert_array_equal(o_ids[0], np.arange(len(sel)))
        ids[t, :len(sel)], wts[t, :len(sel)] = sel, o_w[0]
    x64 = host(x.double())
    xq, _ = moe.quantize_activation(x64, layer.a_fmt) if layer.input_scale is None else \
        _static(x64, float(layer.input_scale))
    pairs = [(t, j) for t in range(T) for j in range(k) if ids[t, j] >= 0]
    h = np.zeros((len(pairs), I))
    ts = lambda s, e: None if s is None else s[e]
    for p, (t, j) in enumerate(pairs):
        e = ids[t, j]
        gu = _deq(layer.w13[e], layer.w13_scale[e], ts(layer.w13_scale_2, e), layer.w_fmt) @ xq[t]
        h[p] = moe.silu(gu[:I]) * gu[I:]
    if pairs:
        h, _ = moe.quantize_activation(h, layer.a_fmt) if layer.inter_scale is None else _static(h, float(layer.inter_scale))
    y = np.zeros((T, layer.hidden))
    for p, (t, j) in enumerate(pairs):
        e = ids[t, j]
        y[t] += float(wts[t, j]) * (_deq(layer.w2[e], layer.w2_scale[e], ts(layer.w2_scale_2, e), layer.w_fmt) @ h[p])
    if layer.shared_inter:
        xs, _ = moe.quantize_activation(x64, "mxfp8")
        gu = xs @ _deq(layer.ws13, layer.ws13_scale, None, "mxfp8").T
        S = layer.shared_inter
        hs, _ = moe.quantize_activation(moe.silu(gu[:, :S]) * gu[:, S:], "mxfp8")
        y += moe.sigmoid(x64 @ host(layer.shared_gate.double()))[:, None] * (hs @ _deq(layer.ws2, layer.ws2_scale, None, "mxfp8").T)
    return ids, wts, y


def _static(v, s):
    from oracle import quant
    q = quant.quantize_nvfp4(v, "rtn", tensor_scale=np.float32(s))
    return quant.dequantize_nvfp4(q["codes"], q["scales"], q["tensor_scale"]), q


def _inputs(T, E, H, seed, ties=False):
    g = _gen(seed)
    x = torch.randn(T, H, device="cuda", generator=g).to(torch.bfloat16)
    lg = torch.randn(T, E, device="cuda", generator=g)
    return x, torch.round(lg * 2) / 2 if ties else lg


def _check(layer, x, lg, bias=None):
    few = _m().FewTokenLayer(layer, int(x.shape[0]))
    y, ids, w = few(x, lg, bias)
    e_ids, e_w, e_y = _expected(layer, x, lg, bias)
    np.testing.assert_array_equal(host(ids), e_ids)
    np.testing.assert_array_max_ulp(host(w), e_w, maxulp=1)
    bar = 1e-5 if layer.a_fmt == "none" and not layer.shared_inter else 2e-3
    err = rel_fro(host(y), e_y) if np.any(e_y) else float(y.abs().max())
    print(f"  rel {err:.2e}", flush=True)
    assert err <= bar
    again, _, _ = few(x, lg, bias)
    assert torch.equal(y, again)
    yb, _, _ = _m().FewTokenLayer(layer, 16, torch.bfloat16)(x, lg, bias)  # another workspace size
    assert torch.equal(yb, y.to(torch.bfloat16))
    return y, ids, w


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("T,E,H,I,k", [(1, 8, 256, 128, 2), (2, 5, 128, 128, 5), (3, 64, 640, 256, 4), (5, 40, 1280, 384, 10),
                                       (8, 16, 384, 640, 3), (16, 24, 512, 128, 6), (11, 130, 256, 256, 7)])
def test_modes_and_sizes(mode, T, E, H, I, k):
    print_case(f"few {mode} T={T} E={E} H={H} I={I} k={k}")
    layer = _layer(mode, E, H, I, k, seed=T * 31 + E)
    x, lg = _inputs(T, E, H, seed=T + E)
    _check(layer, x, lg, torch.randn(E, device="cuda", generator=_gen(4)) if T % 2 else None)


@pytest.mark.parametrize("mode", ["nv", "mx"])
@pytest.mark.parametrize("T,E,H,I,k", [(1, 1, 32, 32, 1), (4, 3, 96, 32, 2), (7, 9, 160, 96, 4), (2, 6, 2592, 672, 3),
                                       (16, 4, 4000, 160, 2), (3, 7, 1056, 1024, 2), (1, 12, 4096, 64, 12)])
def test_widths_that_end_inside_a_step(mode, T, E, H, I, k):
    print_case(f"few ragged {mode} T={T} E={E} H={H} I={I} k={k}")
    _check(_layer(mode, E, H, I, k, seed=H + I), *_inputs(T, E, H, seed=T))


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("T,S", [(1, 128), (6, 384), (16, 1280)])
def test_shared_expert(mode, T, S):
    print_case(f"few shared {mode} T={T} S={S}")
    layer = _layer(mode, 12, 512, 256, 3, seed=S, shared=S)
    _check(layer, *_inputs(T, 12, 512, seed=S + T))


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("shared", [0, 128])
def test_masked_experts_and_empty_slots(mode, shared):
    """-inf logits: fewer experts than k, tokens with none (first, middle and last), all tokens with none."""
    print_case(f"few masked {mode} shared={shared}")
    E, H, I, k = 10, 256, 128, 4
    layer = _layer(mode, E, H, I, k, seed=8, shared=shared)
    x, lg = _inputs(7, E, H, seed=3)
    lg[0] = lg[3] = lg[6] = float("-inf")
    lg[1, 2:] = float("-inf")
    lg[2, 1:] = float("-inf")
    lg[4, ::2] = float("-inf")
    y, ids, w = _check(layer, x, lg)
    assert bool((ids[0] == -1).all()) and bool((w[3] == 0).all()) and int((ids[1] >= 0).sum()) == 2
    if not shared:
        assert float(y[[0, 3, 6]].abs().max()) == 0.0
    lg[:] = float("-inf")
    y, ids, _ = _check(layer, x, lg)
    assert bool((ids == -1).all())
    bias = torch.zeros(E, device="cuda")
    bias[3:] = float("-inf")  # experts masked by the bias
    _check(layer, x, _inputs(7, E, H, seed=4)[1], bias)


@pytest.mark.parametrize("E,k", [(8, 3), (64, 32), (65, 32), (129, 5), (300, 10), (513, 10), (1024, 32)])
def test_routing_ties_and_widths(E, k):
    print_case(f"few routing E={E} k={k}")
    layer = _layer("mx", E, 64, 32, k, seed=E)
    x, lg = _inputs(16, E, 64, seed=E + k, ties=True)
    lg[3] = 0.0
    lg[4] = -0.0
    lg[4, 1::2] = 0.0
    lg[5] = torch.where(lg[5] > 0.4, lg[5], torch.full_like(lg[5], float("-inf")))
    _check(layer, x, lg)
    ids, w = _m().route(lg[:5].contiguous(), k)
    _, ids2, w2 = _m().FewTokenLayer(layer, 5)(x[:5].contiguous(), lg[:5].contiguous())
    assert torch.equal(ids, ids2) and torch.allclose(w, w2, rtol=2.0 ** -22, atol=0)


def test_nan_stays_in_its_token():
    """A NaN or infinite x spoils its own row of y only; a NaN logit is never selected."""
    print_case("few nan")
    layer = _layer("nv", 6, 128, 64, 2, seed=2)
    x, lg = _inputs(4, 6, 128, seed=9)
    ref, ids, _ = _m().FewTokenLayer(layer, 4)(x, lg)
    x2 = x.clone()
    x2[1, 5] = float("nan")
    x2[3, 7] = float("inf")
    y, _, _ = _m().FewTokenLayer(layer, 4)(x2, lg)
    assert torch.equal(y[[0, 2]], ref[[0, 2]]) and bool(torch.isnan(y[1]).any()) and not bool(torch.isfinite(y[3]).all())
    lg2 = lg.clone()
    lg2[0, int(ids[0, 0])] = float("nan")
    lg3 = lg.clone()
    lg3[0, int(ids[0, 0])] = float("-inf")
    a, b = _m().FewTokenLayer(layer, 4)(x, lg2), _m().FewTokenLayer(layer, 4)(x, lg3)
    assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_static_scales():
    print_case("few static NVFP4 scales")
    layer = _layer("nvnv", 8, 256, 128, 2, seed=6)
    layer.input_scale = torch.tensor([4.5 / 2688], device="cuda")
    layer.inter_scale = torch.tensor([3.0 / 2688], device="cuda")
    _check(layer, *_inputs(5, 8, 256, seed=1))


@pytest.mark.parametrize("mode", MODES)
def test_agrees_with_the_layer_forward(mode):
    """Same layer through moe_route + moe_forward (other kernels): within the sum of both bars."""
    print_case(f"few vs forward {mode}")
    m = _m()
    layer = _layer(mode, 32, 512, 256, 4, seed=12, shared=128)
    x, lg = _inputs(9, 32, 512, seed=2)
    y, ids, w = m.FewTokenLayer(layer, 9)(x, lg)
    r_ids, r_w = m.route(lg, 4)
    assert torch.equal(ids, r_ids)
    assert rel_fro(host(y), host(m.moe_forward(layer, x, r_ids, r_w))) <= 4e-3


@pytest.mark.parametrize("mode", MODES)
def test_nothing_outside_the_outputs_is_written(mode):
    print_case(f"few canary {mode}")
    layer = _layer(mode, 8, 256, 128, 3, seed=3, shared=128)
    x, lg = _inputs(3, 8, 256, seed=5)
    for out in (torch.float32, torch.bfloat16):
        few = _m().FewTokenLayer(layer, 3, out)
        need = few.workspace.numel()
        few.workspace = torch.full((need + 4096,), 171, dtype=torch.uint8, device="cuda")[:need]
        tail = torch.as_strided(few.workspace, (4096,), (1,), need)
        buf = torch.full((3 * 256 + 2048,), -7.0, dtype=out, device="cuda")
        iw = torch.full((9 + 512,), -7, dtype=torch.int32, device="cuda")
        ww = torch.full((9 + 512,), -7.0, device="cuda")
        y, ids, w = few(x, lg, None, buf[1024:1024 + 768].view(3, 256), iw[256:265].view(3, 3), ww[256:265].view(3, 3))
        ref = _m().FewTokenLayer(layer, 3, out)(x, lg)
        assert torch.equal(y, ref[0]) and torch.equal(ids, ref[1]) and torch.equal(w, ref[2])
        assert bool((buf[:1024] == -7).all()) and bool((buf[1024 + 768:] == -7).all())
        assert bool((iw[:256] == -7).all()) and bool((iw[265:] == -7).all())
        assert bool((ww[:256] == -7).all()) and bool((ww[265:] == -7).all())
        assert bool((tail == 171).all())
    y, ids, w = few(x[:0], lg[:0])
    assert y.shape == (0, 256) and ids.shape == (0, 3)


def test_streams_and_captured_graphs():
    """A side stream, and two graphs with a workspace each replayed in turns on new inputs (another
    number of touched experts in each) with eager work between."""
    print_case("few graphs")
    m = _m()
    runs = []
    for mode, T in (("nv", 3), ("mxmx", 16), ("nvnv", 5)):
        layer = _layer(mode, 20, 256, 128, 3, seed=T, shared=128 if T == 16 else 0)
        x, lg = _inputs(T, 20, 256, seed=T)
        eager, few = m.FewTokenLayer(layer, T), m.FewTokenLayer(layer, T)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            side = few(x, lg)
        torch.cuda.current_stream().wait_stream(s)
        for a, b in zip(side, eager(x, lg)):
            assert torch.equal(a, b)
        out = tuple(torch.empty_like(v) for v in side)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            few(x, lg, None, *out)
        runs.append((eager, x, lg, out, gr, few))  # the graph works in few's workspace
    for rep in range(4):
        for eager, x, lg, out, gr, _ in runs:
            x.copy_(torch.roll(x, 3, dims=1))
            lg.copy_(torch.roll(lg, 1 + rep, dims=1))
            if rep == 2:
                lg[0] = float("-inf")
            gr.replay()
            for a, b in zip(out, eager(x, lg)):
                assert torch.equal(a, b), rep
        torch.cuda.synchronize()


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("T,E,H,I,k", [(1, 4, 256, 2304, 2), (16, 3, 128, 2304, 2), (6, 9, 384, 1280, 4), (16, 200, 128, 1152, 3)])
def test_wide_intermediates(mode, T, E, H, I, k):
    """K of the down products in several segments, many pairs of an expert in several passes."""
    print_case(f"few wide {mode} T={T} E={E} H={H} I={I} k={k}")
    _check(_layer(mode, E, H, I, k, seed=I + T), *_inputs(T, E, H, seed=E))


@pytest.mark.parametrize("mode", ["nv", "nvnv", "mx", "mxmx"])
@pytest.mark.parametrize("at", [2, 4, 12])
@pytest.mark.parametrize("H,I", [(512, 256), (256, 128), (384, 384)])
def test_scales_at_any_alignment(mode, at, H, I):
    """Block scales that begin `at` bytes behind a multiple of 16 give the same bits."""
    print_case(f"few scales at {at} {mode}")
    layer = _layer(mode, 6, H, I, 2, seed=at)
    x, lg = _inputs(3, 6, H, seed=at)
    ref = _m().FewTokenLayer(layer, 3)(x, lg)
    for name in ("w13_scale", "w2_scale"):
        t = getattr(layer, name)
        room = torch.zeros(t.numel() + 64, dtype=torch.uint8, device="cuda")
        off = (at - room.data_ptr()) % 16
        moved = room[off:off + t.numel()].view(t.dtype).view(t.shape)
        moved.copy_(t)
        setattr(layer, name, moved)
    for a, b in zip(ref, _m().FewTokenLayer(layer, 3)(x, lg)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("sx,sh", [(0.25, 0.5), (2.0 ** -6, 2.0 ** -6), (700.0, 40.0), (1e-12, 1e-19), (2.0 ** -9 * 6, 100.0)])
def test_static_scales_that_clip_and_tie(sx, sh):
    """Tensor scales far from the data's (clipped blocks, subnormal and zero block scales), powers of
    two with x on a grid of quarters (values at the borders between codes)."""
    print_case(f"few static NVFP4 scales {sx} {sh}")
    layer = _layer("nvnv", 8, 256, 128, 2, seed=6)
    layer.input_scale = torch.tensor([sx / 6], device="cuda")
    layer.inter_scale = torch.tensor([sh / 6], device="cuda")
    x, lg = _inputs(5, 8, 256, seed=1)
    x[::2] = torch.round(x[::2] * 4) / 4
    x[1, :32] = 0.0
    _check(layer, x, lg)


def test_one_layer_for_every_count_of_tokens():
    """One workspace, 1 to 16 tokens in turn: each call as if alone."""
    print_case("few counts")
    for mode in MODES:
        layer = _layer(mode, 30, 256, 128, 3, seed=1, shared=256)
        x, lg = _inputs(16, 30, 256, seed=2)
        few = _m().FewTokenLayer(layer, 16)
        for T in (16, 1, 9, 8, 2, 15, 3):
            xs, ls = x[:T].contiguous(), lg[:T].contiguous()
            for a, b in zip(few(xs, ls), _m().FewTokenLayer(layer, T)(xs, ls)):
                assert torch.equal(a, b), (mode, T)
