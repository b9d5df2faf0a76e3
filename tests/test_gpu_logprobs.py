"""token_logprobs and token_logprobs_grad against their definitions in float64.

Tolerances (f32 arithmetic, u = 2^-24): z = (l - M) / T is off by 3 u |z| (difference,
1 / T, product), e^z by that and 4 u relatively, and a sum by u for each addition that
a value passes through, A of them: V / 256 + 80 at most (256 threads a row, or more
of them).  With R = Z - 1, Ez = sum p |z|, Ezz = sum p z^2, each against the definition:
  R          dR = u (3 Ez Z + (A + 4) R)
  ln Z       dL = dR / Z + 2 u ln Z
  logprob    dL + u (3 |z_t| + |logprob|)
  entropy    dH = dL + u (3 Ezz + (A + 10) Ez) + Ez dR / Z + 2 u H
  gradient   of p: p (u (3 |z| + 8) + dR / Z); of 1 - p_t: dR / Z + u (3 |z_t| p_t + 8 (1 - p_t)); of ln p + H:
             u (5 |z| + 4 ln Z + 2 H) + dL + dH; then half a step of the result's type
Over all rows the additions' errors are random: the norm of the errors stays within
the norm of these tolerances with 2 sqrt(A) in A's place."""
import math

import pytest

from gpu_util import gpu_ok, print_case, torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_ok(), reason="needs a GPU")]

from head_util import INF, gen, logprobs64  # noqa: E402

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _m():
    import block_scaled_fp4_nvfp4_amd as m
    return m


def _logits(g, T, V, dtype, scale=3.0, pad=0):
    return (torch.randn(T, V + pad, device="cuda", generator=g) * scale).to(dtype)[:, :V]


def _row(ref, i, A):
    """(Ez, lnZ, dR, dL, dH) of row i."""
    lp, R, Z = ref["lp"][i], ref["R"][i], ref["Z"][i]
    left = lp > -INF
    lnZ = math.log1p(R)
    z, p = lp[left] + lnZ, torch.exp(lp[left])
    Ez, Ezz = float((p * z.abs()).sum()), float((p * z * z).sum())
    dR = U * (3 * Ez * Z + (A + 4) * R)
    dL = dR / Z + 2 * U * lnZ
    return Ez, lnZ, dR, dL, dL + U * (3 * Ezz + (A + 10) * Ez) + Ez * dR / Z + 2 * U * ref["entropy"][i]


def check(logits, targets, r, temperature=1.0, top=0):
    T, V = logits.shape
    ref = logprobs64(logits, targets, temperature, top)
    A = V / 256 + 80
    stats = r["stats"].tolist()
    if targets is not None:
        assert r["ranks"].tolist() == ref["ranks"]
    if top:
        assert r["top_ids"].tolist() == ref["top_ids"]
    compared = {"R": [], "H": [], "lp": []}  # (got, wanted, tolerance, tolerance of random errors)
    for i in range(T):
        given = targets is not None and 0 <= int(targets[i]) < V
        if targets is not None and not given:
            assert float(r["logprobs"][i]) == 0.0
        lps = ([(float(r["logprobs"][i]), ref["logprobs"][i])] if given else []) + (list(zip(r["top_logprobs"][i].tolist(), ref["top_logprobs"][i])) if top else [])
        assert stats[i][0] == ref["M"][i] and float(r["entropy"][i]) == stats[i][2]
        if ref["Z"][i] == 0:
            assert stats[i] == [-INF, -1.0, 0.0] and all(got == -INF for got, _ in lps)
            continue
        _, lnZ, dR, dL, dH = _row(ref, i, A)
        _, _, sR, sL, sH = _row(ref, i, 2 * A ** 0.5)
        compared["R"].append((stats[i][1], ref["R"][i], dR, sR))
        compared["H"].append((stats[i][2], ref["entropy"][i], dH, sH))
        for got, want in lps:
            if want == -INF:
                assert got == want
            else:
                more = U * (3 * abs(want + lnZ) + abs(want))
                compared["lp"].append((got, want, dL + more, sL + more))
    for name, rows in compared.items():
        if rows:
            got, want, tol, random = torch.tensor(rows, dtype=torch.float64).T
            err = (got - want).abs()
            assert bool((err <= tol + 1e-300).all()), (name, float((err / tol.clamp(min=1e-300)).max()))
            assert float(err.norm()) <= float(random.norm()) + 1e-300, (name, float(err.norm()), float(random.norm()))


SIZES = [(1, 1), (3, 2), (1, 7), (2, 63), (5, 64), (4, 65), (1, 100), (300, 129), (3, 255), (2, 1000), (1, 4095), (7, 4097), (2, 9000), (1, 32000),
         (40, 2049), (3, 33333), (1, 131072), (2, 250001), (600, 520)]


@pytest.mark.parametrize("T,V", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("top", [0, 1, 5, 64])
def test_sizes(T, V, dtype, top):
    print_case(f"logprobs T={T} V={V} {dtype} top={top}")
    g = gen(T + V)
    logits = _logits(g, T, V, DT[dtype])
    targets = torch.randint(0, V, (T,), device="cuda", generator=g).int()
    r = _m().token_logprobs(logits, targets, top=top)
    check(logits, targets, r, top=top)
    again = _m().token_logprobs(logits, targets, top=top)
    assert all(torch.equal(r[k], again[k]) for k in r)


@pytest.mark.parametrize("pad", [1, 3, 8, 72])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("temperature", [0.05, 0.7, 1.3, 40.0])
def test_strides_and_temperatures(pad, dtype, temperature):
    """Rows of a padded head (NaN in the padding), at any alignment."""
    print_case(f"logprobs pad={pad} {dtype} T={temperature}")
    g = gen(pad)
    for T, V in ((3, 1001), (1, 5000), (2, 40007)):
        base = torch.full((T * (V + pad) + 1,), float("nan"), device="cuda", dtype=DT[dtype])
        logits = base[1:].view(T, V + pad)[:, :V]
        logits.copy_(_logits(g, T, V, DT[dtype]))
        targets = torch.randint(0, V, (T,), device="cuda", generator=g).int()
        r = _m().token_logprobs(logits, targets, top=7, temperature=temperature)
        check(logits, targets, r, temperature, 7)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [50, 3000, 70001])
def test_masks_ties_and_order(dtype, V):
    """Rows with everything masked, one token left, all equal, in rising and falling order, many ties, the
    lowest values of the type, a target that is masked, out of range, or missing."""
    print_case(f"logprobs masks {dtype} V={V}")
    g = gen(V)
    T = 12
    logits = _logits(g, T, V, DT[dtype])
    logits[0] = -INF
    logits[1] = -INF
    logits[1, V // 2] = 2.0
    logits[2] = 1.5
    logits[3] = torch.linspace(-9, 9, V, device="cuda").to(DT[dtype])
    logits[4] = torch.linspace(9, -9, V, device="cuda").to(DT[dtype])
    logits[5] = torch.randint(0, 3, (V,), device="cuda", generator=g).to(DT[dtype])
    logits[6, torch.rand(V, device="cuda", generator=g) < 0.95] = -INF
    logits[6, 3] = 0.0
    logits[7] = torch.finfo(DT[dtype]).min
    logits[7, V - 1] = 0.0
    logits[8] = torch.finfo(DT[dtype]).min
    logits[9] = 300.0
    logits[9, 0] = -300.0
    logits[10, 2:] = -INF
    targets = torch.tensor([3, V // 2, 7, V - 1, 0, V // 3, 3, 5, V - 1, 0, V - 1, -1], device="cuda", dtype=torch.int32)
    for top in (0, 20, 64):
        r = _m().token_logprobs(logits, targets, top=top)
        check(logits, targets, r, top=top)
    targets[11] = V
    check(logits, targets, _m().token_logprobs(logits, targets, top=3), top=3)
    targets[11] = -2 ** 31
    check(logits, targets, _m().token_logprobs(logits, targets))
    r = _m().token_logprobs(logits, None, top=2)
    assert set(r) == {"entropy", "stats", "top_ids", "top_logprobs"}
    check(logits, None, r, top=2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [70, 20000])
def test_not_finite(dtype, V):
    """NaN and +inf make their own row NaN and no other; a NaN is never an alternative."""
    print_case(f"logprobs NaN {dtype} V={V}")
    g = gen(V)
    logits = _logits(g, 4, V, DT[dtype])
    clean = logits.clone()
    logits[0, V // 2] = float("nan")
    logits[2, V - 1] = INF
    targets = torch.zeros(4, device="cuda", dtype=torch.int32)
    r, c = _m().token_logprobs(logits, targets, top=5), _m().token_logprobs(clean, targets, top=5)
    for key in ("logprobs", "entropy"):
        assert torch.isnan(r[key]).tolist() == [True, False, True, False]
    for key in r:
        assert torch.equal(r[key][1::2], c[key][1::2])
    finite = logits[0].float().nan_to_num(nan=-INF)
    assert r["top_ids"][0].tolist() == torch.sort(finite, descending=True, stable=True).indices[:5].tolist()
    assert int(r["top_ids"][2, 0]) == V - 1
    d = _m().token_logprobs_grad(logits, targets, r["stats"], torch.ones(4, device="cuda"))
    assert torch.isnan(d).all(1).tolist() == [True, False, True, False]


def grad64(logits, targets, temperature, glp, gH):
    """(gradient, tolerance) in float64."""
    ref = logprobs64(logits, targets, temperature)
    T, V = logits.shape
    d, tol = torch.zeros(T, V, dtype=torch.float64), torch.zeros(T, V, dtype=torch.float64)
    for i in range(T):
        if ref["Z"][i] == 0:
            continue
        lp, H, Z = ref["lp"][i], ref["entropy"][i], ref["Z"][i]
        p = torch.exp(lp)
        t = int(targets[i])
        a = float(glp[i]) if glp is not None and 0 <= t < V else 0.0
        b = float(gH[i]) if gH is not None else 0.0
        _, lnZ, dR, dL, dH = _row(ref, i, V / 256 + 80)
        inner = torch.where(p > 0, lp + H, torch.zeros_like(p))
        z = torch.where(p > 0, (lp + lnZ).abs(), torch.zeros_like(p))
        dp = p * (U * (3 * z + 8) + dR / Z)
        d[i] = -a * p - b * p * inner
        tol[i] = abs(a) * dp + abs(b) * (dp * inner.abs() + p * (U * (5 * z + 4 * lnZ + 2 * H) + dL + dH)) + 4 * U * d[i].abs()
        if a:
            q = -float(torch.expm1(lp[t]))
            d[i, t] += a * (q + float(p[t]))
            tol[i, t] += abs(a) * (dR / Z + U * (3 * float(z[t]) * float(p[t]) + 8 * q))
    return d / temperature, tol / temperature


@pytest.mark.parametrize("T,V", [(1, 1), (3, 7), (2, 64), (5, 129), (300, 130), (1, 1000), (2, 4097), (3, 33333), (1, 131072), (40, 2050)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("which", ["logprob", "entropy", "both"])
def test_gradients(T, V, dtype, which):
    print_case(f"logprobs grad T={T} V={V} {dtype} {which}")
    g = gen(T * V)
    temperature = 0.8 if which == "both" else 1.0
    logits = _logits(g, T, V, DT[dtype], pad=V % 3)
    if V > 1:
        logits[T - 1, torch.rand(V, device="cuda", generator=g) < 0.5] = -INF
        logits[T - 1, V // 2] = 1.0
    targets = torch.randint(0, V, (T,), device="cuda", generator=g).int()
    if T > 2:
        targets[1] = -1
    glp = torch.randn(T, device="cuda", generator=g) if which != "entropy" else None
    gH = torch.randn(T, device="cuda", generator=g) if which != "logprob" else None
    stats = _m().token_logprobs(logits, targets, temperature=temperature)["stats"]
    d = _m().token_logprobs_grad(logits, targets if glp is not None else None, stats, glp, gH, temperature)
    assert d.dtype == logits.dtype and d.shape == (T, V)
    e, tol = grad64(logits, targets, temperature, glp, gH)
    tol = tol + torch.finfo(DT[dtype]).eps / 2 * e.abs() + torch.finfo(DT[dtype]).smallest_normal * 2.0 ** -7
    bad = ~((d.double().cpu() - e).abs() <= tol)
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:3].tolist())
    # in the logits' own memory, and into rows at a stride of their own, whose padding stays as it was
    own = logits.clone()
    base = torch.full((T, V + 5), 9.0, device="cuda", dtype=DT[dtype])
    assert torch.equal(_m().token_logprobs_grad(own, targets, stats, glp, gH, temperature, out=own), d)
    _m().token_logprobs_grad(logits, targets, stats, glp, gH, temperature, out=base[:, 2:2 + V])
    assert torch.equal(base[:, 2:2 + V], d) and bool((base[:, :2] == 9.0).all()) and bool((base[:, 2 + V:] == 9.0).all())


@pytest.mark.parametrize("V", [5, 700])
def test_gradient_against_differences(V):
    """Central differences of the kernel's own outputs: step h = 2^-6 leaves h^2 / 6 of the third derivative (below 2 for
    both) and the values' rounding, 16 ulp of at most 8, over h."""
    print_case(f"logprobs differences V={V}")
    g = gen(V)
    logits = _logits(g, 1, V, torch.float32, 1.0)
    targets = torch.tensor([V // 2], device="cuda", dtype=torch.int32)
    h, temperature = 2.0 ** -6, 0.9
    glp, gH = torch.tensor([0.7], device="cuda"), torch.tensor([-1.3], device="cuda")
    stats = _m().token_logprobs(logits, targets, temperature=temperature)["stats"]
    d = _m().token_logprobs_grad(logits, targets, stats, glp, gH, temperature)[0]
    js = torch.arange(V, device="cuda") if V < 100 else torch.tensor([0, 1, V // 2, V - 1], device="cuda")
    step = torch.zeros(len(js), V, device="cuda")
    step[torch.arange(len(js), device="cuda"), js] = h
    value = lambda l: (lambda r: 0.7 * r["logprobs"].double() - 1.3 * r["entropy"].double())(  # noqa: E731
        _m().token_logprobs(l, targets.expand(len(js)).contiguous(), temperature=temperature))
    diff = (value(logits + step) - value(logits - step)) / (2 * h)
    assert float((d[js].double() - diff).abs().max()) <= 2 * (h / temperature) ** 2 / temperature + 16 * 8 * U / h


def test_no_rows():
    fp = _m()
    r = fp.token_logprobs(torch.empty(0, 50, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"), top=3)
    assert r["top_ids"].shape == (0, 3) and r["logprobs"].shape == (0,)
    assert fp.token_logprobs_grad(torch.empty(0, 50, device="cuda"), None, r["stats"], None).shape == (0, 50)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(2, 1001), (3, 70001), (800, 3001)])
def test_temperatures_at_the_ends(dtype, T, V):
    """The least temperature leaves the largest logit alone, a huge one makes all tokens alike."""
    print_case(f"logprobs T={T} V={V} {dtype}, temperatures 2^-100 and 2^126")
    g = gen(V)
    logits = _logits(g, T, V, DT[dtype]).clamp(-50, 50)
    best = torch.randint(0, V, (T,), device="cuda", generator=g)
    other = (best + 1) % V
    rows = torch.arange(T, device="cuda")
    logits[rows, best] = 64.0
    glp, gH = torch.ones(T, device="cuda"), torch.full((T,), -0.5, device="cuda")
    cold = 2.0 ** -100
    r = _m().token_logprobs(logits, best.int(), top=2, temperature=cold)
    assert bool((r["logprobs"] == 0).all()) and bool((r["entropy"] == 0).all()) and bool((r["ranks"] == 0).all())
    assert torch.equal(r["top_ids"][:, 0].long(), best) and bool((r["top_logprobs"][:, 1] <= -14 * 2.0 ** 100 * (1 - 2.0 ** -20)).all())
    d = _m().token_logprobs_grad(logits, best.int(), r["stats"], glp, gH, cold)
    assert bool((d == 0).all())
    # another target: -p_best / T at the largest logit, 1 / T at the target
    d = _m().token_logprobs_grad(logits, other.int(), r["stats"], glp, gH, cold).float()
    assert bool((d[rows, best] == -1 / cold).all()) and bool((d[rows, other] == 1 / cold).all()) and int((d != 0).sum()) == 2 * T
    r = _m().token_logprobs(logits, best.int(), temperature=2.0 ** 126)
    lnv = math.log(V)
    # every exponential is 1 and Z - 1 exact; log1p and one rounding
    assert float((r["logprobs"] + lnv).abs().max()) <= 4 * 2.0 ** -24 * lnv and float((r["entropy"] - lnv).abs().max()) <= 4 * 2.0 ** -24 * lnv
    d = _m().token_logprobs_grad(logits, best.int(), r["stats"], glp, gH, 2.0 ** 126)
    assert bool((d.abs() <= 2.0 ** -126).all())
