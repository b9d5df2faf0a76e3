"""token_logprobs and token_logprobs_grad with very many rows, and rows of very many logits."""
import pytest

from gpu_util import gpu_ok, print_case, torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_ok(), reason="needs a GPU")]

from head_util import gen  # noqa: E402

U = 2.0 ** -24


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_million_rows(dtype):
    """Few values are added up (A = 80 at most); |z| < 40 in logits of at most 20, H < 4: all errors within 400 u (1 + |ln p|)."""
    import block_scaled_fp4_nvfp4_amd as fp
    T, V = (1 << 20) + 3, 33
    print_case(f"logprobs T={T} V={V} {dtype}")
    g = gen(1)
    logits = (torch.randn(T, V, device="cuda", generator=g) * 2).clamp(-10, 10).to(dtype)
    targets = torch.randint(0, V, (T,), device="cuda", generator=g).int()
    r = fp.token_logprobs(logits, targets, top=2)
    l64, t = logits.double(), targets.long()[:, None]
    lp = torch.log_softmax(l64, 1)
    own = lp.gather(1, t)[:, 0]
    assert bool(((r["logprobs"].double() - own).abs() <= 400 * U * (1 + own.abs())).all())
    H = -(lp.exp() * lp).sum(1)
    assert bool(((r["entropy"].double() - H).abs() <= 400 * U * (1 + H) ** 2).all())
    lt = l64.gather(1, t)
    ids = torch.arange(V, device="cuda")[None]
    assert torch.equal(r["ranks"].long(), ((l64 > lt) | ((l64 == lt) & (ids < t))).sum(1))
    assert torch.equal(r["top_ids"].long(), torch.sort(l64, dim=1, descending=True, stable=True).indices[:, :2])
    one = torch.ones(T, device="cuda")
    d = fp.token_logprobs_grad(logits, targets, r["stats"], one)
    want = torch.zeros_like(lp).scatter_(1, t, 1.0) - lp.exp()
    assert bool(((d.double() - want).abs() <= 400 * U + torch.finfo(dtype).eps / 2 * want.abs()).all())


def test_rows_of_2_to_the_28():
    """Two rows, 64 parts each, whose 256 lanes add up V / 2^14 values; ids and ranks are exact.  A value of a sum passes A = 2^14
    + 80 additions of u at most."""
    import block_scaled_fp4_nvfp4_amd as fp
    T, V = 2, (1 << 28) + 5
    print_case(f"logprobs T={T} V={V}")
    g = gen(2)
    logits = torch.randn(T, V, device="cuda", generator=g).clamp_(-8, 8).bfloat16()
    for at, value in ((V - 1, 20.0), (7, 19.0), (V // 2, 19.0), (V - 3, 12.0)):
        logits[0, at] = value
    logits[1, V - 2] = 9.0
    targets = torch.tensor([V // 2, V - 1], dtype=torch.int32, device="cuda")
    r = fp.token_logprobs(logits, targets, top=4)
    assert r["top_ids"][0].tolist() == [V - 1, 7, V // 2, V - 3] and int(r["top_ids"][1, 0]) == V - 2
    A = 2 ** 14 + 80
    for i in range(T):
        l = logits[i]
        t, M = int(targets[i]), float(l.max())
        Z = sum(float(torch.exp(part.double() - M).sum()) for part in l.split(1 << 26))
        E = sum(float((torch.exp(part.double() - M) * (M - part.double())).sum()) for part in l.split(1 << 26))
        assert int(r["ranks"][i]) == int((l > l[t]).sum()) + int((l[:t] == l[t]).sum())
        dL = U * (3 * E / Z + A + 4) + 4 * U * 25
        lnZ = float(torch.tensor(Z, dtype=torch.float64).log())
        assert abs(float(r["logprobs"][i]) - (float(l[t]) - M - lnZ)) <= dL + 4 * U * 40
        assert abs(float(r["entropy"][i]) - (lnZ + E / Z)) <= dL + U * (2 * A + 3 * 40) * E / Z
    one = torch.ones(T, device="cuda")
    d = fp.token_logprobs_grad(logits, targets, r["stats"], one)
    for i in range(T):
        t = int(targets[i])
        for at in (0, t - 1, t, V - 1, V - 2):
            p = float(torch.exp(logits[i, at].double() - float(r["stats"][i, 0]))) / (1 + float(r["stats"][i, 1]))
            want = (1.0 if at == t else 0.0) - p
            assert abs(float(d[i, at]) - want) <= 2.0 ** -8 * abs(want) + 400 * U * p
