"""The 4-bit head and what is read from it, run together as a training step and a
decode step use them: hidden states -> fp4_matmul -> logits -> token_logprobs ->
token_logprobs_grad -> fp4_matmul_grad -> gradient of the hidden states; on two
streams at once, captured and replayed, in poisoned workspaces, at offsets beyond
32 bits."""
import pytest

from gpu_util import gpu_ok, print_case, torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_ok(), reason="needs a GPU")]

from head_util import INF, gen, raw_weight, w64  # noqa: E402

U = 2.0 ** -24


def _m():
    import block_scaled_fp4_nvfp4_amd as m
    return m


def _head(g, fmt, n, k):
    return _m().quantize(torch.randn(n, k, device="cuda", generator=g) * 0.1, fmt)


def _step(x, w, fmt, V, targets, glp, gH, temperature):
    """One step; the logits' gradient takes the logits' place, the padding of the head has gradient 0."""
    fp = _m()
    logits = fp.fp4_matmul(x, w, fmt, out_dtype=torch.float32)
    r = fp.token_logprobs(logits[:, :V], targets, top=4, temperature=temperature)
    kept = logits[:, :V].clone()
    fp.token_logprobs_grad(logits[:, :V], targets, r["stats"], glp, gH, temperature, out=logits[:, :V])
    logits[:, V:].zero_()
    dx = fp.fp4_matmul_grad(logits, w, fmt, out_dtype=torch.float32)
    return {"logits": kept, "dx": dx, **r}


@pytest.mark.parametrize("T,V,n,k", [(1, 500, 512, 256), (16, 4090, 4096, 640), (70, 1000, 1001, 320), (300, 2000, 2016, 128)])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_training_step(T, V, n, k, fmt):
    """Log probabilities, entropies and the hidden states' gradient against the same step in float64 (autograd).

    With the logits off by d (their sums' rounding, (k + 16) 2^-23 P as in head_util), a log probability or an entropy
    moves by 2 d / temperature (the entropy by d (1 + max |ln p|)); the gradient of the logits moves by no more than
    d (|glp| + |gH| (2 + max |ln p|)) / temperature^2, and by f32's own rounding of p, ln Z and H (200 u
    in all at these sizes: V / 256 + 80 additions); each of these times sum |W| over a column bounds dx."""
    print_case(f"step T={T} V={V} n={n} k={k} {fmt}")
    g = gen(T + n)
    w = _head(g, fmt, n, k)
    x = torch.randn(T, k, device="cuda", generator=g).bfloat16()
    targets = torch.randint(0, V, (T,), device="cuda", generator=g).int()
    glp, gH, temperature = torch.randn(T, device="cuda", generator=g), torch.randn(T, device="cuda", generator=g), 0.9
    r = _step(x, w, fmt, V, targets, glp, gH, temperature)
    rec = {"codes": w["codes"][None], "scales": w["scales"][None], "tensor_scale": w["tensor_scale"]}
    W = w64(rec, fmt)[0]
    xd = x.double().requires_grad_()
    lp = torch.log_softmax((xd @ W.t().contiguous())[:, :V] / temperature, 1)
    chosen = lp.gather(1, targets[:, None].long())[:, 0]
    H = -(lp.exp() * lp).sum(1)
    (glp.double() * chosen + gH.double() * H).sum().backward()
    lp, chosen, H = lp.detach(), chosen.detach(), H.detach()
    d = ((k + 16) * 2.0 ** -23 * (x.double().abs() @ W.abs().t().contiguous())).max()
    most = lp.abs().max()
    assert float((r["logprobs"].double() - chosen).abs().max()) <= float(2 * d / temperature + 400 * U * (1 + most))
    assert float((r["entropy"].double() - H).abs().max()) <= float(d * (1 + most) / temperature + 400 * U * (1 + most) ** 2)
    rank = (lp > chosen[:, None]).sum(1)
    assert int((r["ranks"] - rank).abs().max()) <= 1 + V // 200  # neighbours within the logits' rounding may change places
    move = (glp.abs() + gH.abs() * (2 + most))[:, None] * (d / temperature ** 2 + 400 * U * (1 + most)) + 0 * r["dx"]
    assert bool(((r["dx"].double() - xd.grad).abs() <= move * W.abs().sum(0)).all())
    # over all values these errors are independent: a hundredth of the bound in the Frobenius norm
    assert float((r["dx"].double() - xd.grad).norm()) <= 1e-2 * float((move * W.abs().sum(0)).norm())


def _same(a, b):
    return all(torch.equal(a[key], b[key]) for key in a)


@pytest.mark.parametrize("T,V,n,k", [(1, 32000, 32000, 256), (16, 4090, 4096, 640), (200, 1000, 1001, 336)])
def test_captured_and_replayed(T, V, n, k):
    """The step as a graph, replayed with new inputs between eager steps and other work, against the eager step."""
    print_case(f"graph T={T} n={n} k={k}")
    g = gen(n)
    w = _head(g, "nvfp4", n, k)
    make = lambda: (torch.randn(T, k, device="cuda", generator=g).bfloat16(), torch.randint(0, V, (T,), device="cuda", generator=g).int(),  # noqa: E731
                    torch.randn(T, device="cuda", generator=g))
    still = make()
    run = lambda i: _step(i[0], w, "nvfp4", V, i[1], i[2], i[2], 1.1)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(still)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(still)
    for _ in range(4):
        new = make()
        eager = run(new)
        for a, b in zip(still, new):
            a.copy_(b)
        graph.replay()
        other = torch.randn(512, 512, device="cuda") @ torch.randn(512, 512, device="cuda")
        torch.cuda.synchronize()
        assert _same(eager, out)
        del other


def test_two_streams_at_once():
    """Two steps with different sizes on two streams, over and over, against each alone."""
    print_case("two streams")
    g = gen(3)
    jobs = []
    for T, V, n, k in ((16, 30000, 30016, 640), (150, 5000, 5003, 336)):
        w = _head(g, "nvfp4", n, k)
        jobs.append((torch.randn(T, k, device="cuda", generator=g).bfloat16(), w, "nvfp4", V,
                     torch.randint(0, V, (T,), device="cuda", generator=g).int(), torch.randn(T, device="cuda", generator=g),
                     torch.randn(T, device="cuda", generator=g), 1.0))
    alone = [_step(*j) for j in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for st, j in zip(streams, jobs):
            with torch.cuda.stream(st):
                got.append(_step(*j))
        torch.cuda.synchronize()
        assert all(_same(a, b) for a, b in zip(got, alone))


@pytest.mark.parametrize("fill", [0x00, 0xFF, 0x7F])
def test_workspaces_are_written_before_they_are_read(fill):
    fp = _m()
    print_case(f"workspace {fill}")
    g = gen(fill)
    for grad, m, n, k in ((False, 200, 300, 272), (True, 16, 4001, 640), (True, 40, 640, 512)):
        w = raw_weight(g, "nvfp4", 1, n, k)
        x = torch.randn(1, m, n if grad else k, device="cuda", generator=g)
        call = fp.fp4_matmul_grad if grad else fp.fp4_matmul
        size = fp.fp4_matmul_workspace_size(torch.float32, 1, m, n, k, "nvfp4", grad)
        assert size > 0
        space = torch.full((size + 256,), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(call(x, w, "nvfp4", workspace=space[:size]), call(x, w, "nvfp4"))
        assert bool((space[size:] == fill).all())
    logits = torch.randn(3, 300000, device="cuda", generator=g)
    targets = torch.tensor([5, -1, 299999], dtype=torch.int32, device="cuda")
    size = fp.token_logprobs_workspace_size(torch.float32, 3, 300000, 20)
    assert size > 0
    space = torch.full((size + 256,), fill, dtype=torch.uint8, device="cuda")
    assert _same(fp.token_logprobs(logits, targets, top=20, workspace=space[:size]), fp.token_logprobs(logits, targets, top=20))
    assert bool((space[size:] == fill).all())


def test_logits_beyond_32_bits():
    """Rows 2^30 + 8 logits apart: offsets pass 2^31 values and 2^32 bytes."""
    print_case("logits beyond 32 bits")
    fp, V, stride = _m(), 5003, (1 << 30) + 8
    g = gen(1)
    base = torch.empty(2 * stride + V, dtype=torch.bfloat16, device="cuda")
    logits = base.as_strided((3, V), (stride, 1))
    logits.copy_(torch.randn(3, V, device="cuda", generator=g) * 3)
    # rows of the same alignment: which of a row's logits are added up together goes by its 16-byte pieces
    near = torch.empty(3, V + 5, dtype=torch.bfloat16, device="cuda")[:, :V]
    near.copy_(logits)
    targets = torch.tensor([0, V - 1, 7], dtype=torch.int32, device="cuda")
    a, b = fp.token_logprobs(logits, targets, top=5), fp.token_logprobs(near, targets, top=5)
    assert _same(a, b)
    ones = torch.ones(3, device="cuda")
    want = fp.token_logprobs_grad(near, targets, b["stats"], ones, ones)
    fp.token_logprobs_grad(logits, targets, a["stats"], ones, ones, out=logits)
    assert torch.equal(logits, want)


def test_weights_beyond_32_bits():
    """Codes of 2^31 bytes and more: the last rows of W, and their gradient."""
    print_case("weights beyond 32 bits")
    fp, n, k = _m(), (1 << 20) + 48, 4096
    g = gen(2)
    w = {"codes": torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda", generator=g),
         "scales": torch.randint(120, 130, (n, k // 32), dtype=torch.uint8, device="cuda", generator=g)}
    tail = {"codes": w["codes"][-64:].clone(), "scales": w["scales"][-64:].clone()}
    for m in (3, 70):
        x = torch.randn(m, k, device="cuda", generator=g).bfloat16()
        y = fp.fp4_matmul(x, w, "mxfp4", out_dtype=torch.float32)
        e = x.double() @ w64({"codes": tail["codes"][None], "scales": tail["scales"][None]}, "mxfp4")[0].t().contiguous()
        assert float((y[:, -64:].double() - e).norm()) <= 1e-6 * float(e.norm())
        del y
    dy = torch.zeros(2, n, device="cuda", dtype=torch.bfloat16)
    dy[0, n - 1] = 1
    dy[1, n - 60] = -2
    dx = fp.fp4_matmul_grad(dy, w, "mxfp4", out_dtype=torch.float32)
    W = w64({"codes": tail["codes"][None], "scales": tail["scales"][None]}, "mxfp4")[0]
    assert torch.equal(dx.double(), torch.stack((W[63], -2 * W[4])))


def test_decode_step_with_a_grammar():
    """A decode step: f32 logits of 16 sequences, a mask (one sequence finished: nothing left), the likeliest tokens."""
    fp = _m()
    print_case("decode step")
    g = gen(8)
    w = _head(g, "mxfp4", 8192, 256)
    x = torch.randn(16, 256, device="cuda", generator=g).bfloat16()
    logits = fp.fp4_matmul(x, w, "mxfp4", out_dtype=torch.float32)
    logits[:, 4000:] = -INF
    logits[5] = -INF
    r = fp.token_logprobs(logits, None, top=3)
    assert r["top_ids"][5].tolist() == [-1, -1, -1] and int(r["top_ids"].max()) < 4000
    live = [i for i in range(16) if i != 5]
    assert r["top_ids"][live, 0].tolist() == logits[live].argmax(1).tolist()
    again = fp.token_logprobs(logits, r["top_ids"][:, 0].contiguous())
    assert torch.equal(again["logprobs"], r["top_logprobs"][:, 0].masked_fill(r["top_ids"][:, 0] < 0, 0.0))
    assert again["ranks"].tolist() == [0 if i != 5 else -1 for i in range(16)]
