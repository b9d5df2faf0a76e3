"""token_logprobs where a workgroup streams over a row (many rows, or rows too long for its registers): several rounds of
logits a wave, in whole rows and in parts, against float64 (tolerances: test_gpu_logprobs)."""
import math

import pytest

from gpu_util import gpu_ok, print_case, torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_ok(), reason="needs a GPU")]

from head_util import INF, gen, logprobs64  # noqa: E402
from test_gpu_logprobs import DT, check, grad64  # noqa: E402

# 4 waves of 128 pieces of 16 bytes a round: 4096 bf16, 2048 f32 logits.  Parts of a row: 2 of 800 rows, 11 of 100, 32 of 33.
SHAPES = [(800, 20011, 0), (800, 20011, 3), (1100, 9001, 5), (100, 131072, 0), (100, 140003, 1), (33, 600001, 2)]


def _rows(g, T, V, pad, dtype):
    """Logits whose first rows are hard cases."""
    base = torch.full((T * (V + pad) + 1,), float("nan"), device="cuda", dtype=dtype)
    logits = base[1 if pad else 0:][:T * (V + pad)].view(T, V + pad)[:, :V]
    logits.copy_(torch.randn(T, V, device="cuda", generator=g) * 3)
    low = torch.finfo(dtype).min
    ramp = torch.linspace(-9, 9, V, device="cuda")
    steps = (torch.arange(V, device="cuda") // 1500).float()          # a new largest value in every round
    logits[0], logits[1], logits[2], logits[3] = ramp.to(dtype), ramp.flip(0).to(dtype), 1.5, -INF
    logits[4] = -INF
    logits[4, V - 1] = 2.0                                            # all that is left comes last
    logits[5, torch.rand(V, device="cuda", generator=g) < 0.95] = -INF
    logits[6] = torch.randint(0, 3, (V,), device="cuda", generator=g).to(dtype)
    logits[7] = low
    logits[7, V // 3] = 0.0
    logits[8, :V // 2] = -INF
    logits[9] = (steps * 0.05).to(dtype)
    logits[10] = (steps * 4).to(dtype)                                # what came before is all but nothing
    logits[11] = (-steps * 4).to(dtype)
    logits[12] = low
    logits[13, V // 2:] = logits[13, :V - V // 2].clone()             # every value twice, half a row apart
    logits[14, V - 1] = 60.0
    logits[15, 0] = 60.0
    return logits


@pytest.mark.parametrize("T,V,pad", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("top,temperature", [(0, 1.0), (5, 0.7), (64, 1.0)])
def test_rows_of_many_rounds(T, V, pad, dtype, top, temperature):
    import block_scaled_fp4_nvfp4_amd as fp
    print_case(f"logprobs stream T={T} V={V} pad={pad} {dtype} top={top} temperature={temperature}")
    g = gen(T + V + pad)
    logits = _rows(g, T, V, pad, DT[dtype])
    targets = torch.randint(0, V, (T,), device="cuda", generator=g).int()
    targets[:4] = torch.tensor([V - 1, 0, 7, 3])
    targets[5], targets[8], targets[13], targets[14], targets[16] = 1, 0, V - 1, V - 1, -1  # masked ones, late ones, none
    r = fp.token_logprobs(logits, targets, top=top, temperature=temperature)
    sample = torch.tensor(sorted({*range(18), *torch.randint(18, T, (8,), generator=torch.Generator().manual_seed(V)).tolist(), T - 1}), device="cuda")
    got = {k: v[sample] for k, v in r.items()}
    if temperature < 1:  # the type's lowest value, 3.39e38 / 0.7 = 4.8e38 below the largest logit: beyond f32's 3.4028e38, so -inf
        want = logprobs64(logits[sample], targets[sample], temperature, top)
        for key in ("logprobs", "top_logprobs"):
            wanted = torch.tensor(want[key], dtype=torch.float64, device="cuda")
            far = (wanted < -torch.finfo(torch.float32).max) & (wanted > -INF)
            assert bool((got[key][far] == -INF).all()) and bool(far.any())
            got[key] = torch.where(far, wanted, got[key].double())
    check(logits[sample], targets[sample], got, temperature, top)
    again = fp.token_logprobs(logits, targets, top=top, temperature=temperature)
    assert all(torch.equal(r[k], again[k]) for k in r)


@pytest.mark.parametrize("T,V,pad", [(800, 20011, 3), (100, 140003, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_not_finite(T, V, pad, dtype):
    """NaN and +inf, in the first round and the last, make their own row NaN and no other; a NaN is never an alternative."""
    import block_scaled_fp4_nvfp4_amd as fp
    print_case(f"logprobs stream NaN T={T} V={V} {dtype}")
    g = gen(V)
    logits = _rows(g, T, V, pad, DT[dtype])
    clean = logits.clone()
    bad = {20: (0, float("nan")), 22: (V - 1, float("nan")), 24: (V // 2, float("nan")), 26: (3, INF), 28: (V - 1, INF)}
    for row, (at, value) in bad.items():
        logits[row, at] = value
    targets = torch.full((T,), 9, device="cuda", dtype=torch.int32)
    r = fp.token_logprobs(logits, targets, top=5)
    c = fp.token_logprobs(torch.empty_strided(logits.shape, logits.stride(), dtype=logits.dtype, device="cuda").copy_(clean), targets, top=5)
    for key in ("logprobs", "entropy"):
        assert sorted(torch.isnan(r[key]).nonzero()[:, 0].tolist()) == sorted(bad)
    for row in (20, 22, 24):
        assert r["top_ids"][row].tolist() == torch.sort(logits[row].float().nan_to_num(nan=-INF), descending=True, stable=True).indices[:5].tolist()
    for row in (26, 28):
        assert int(r["top_ids"][row, 0]) == bad[row][0]
    good = torch.tensor([i for i in range(T) if i not in bad], device="cuda")
    # the copy's rows lie alike only where its memory starts alike; ids and ranks do not go by that
    assert torch.equal(r["top_ids"][good], c["top_ids"][good]) and torch.equal(r["ranks"][good], c["ranks"][good])


@pytest.mark.parametrize("T,V,pad", [(800, 20011, 3), (2100, 5003, 0), (33, 600001, 2)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_of_many_rows(T, V, pad, dtype):
    import block_scaled_fp4_nvfp4_amd as fp
    print_case(f"logprobs stream grad T={T} V={V} {dtype}")
    g = gen(T)
    logits = _rows(g, T, V, pad, DT[dtype])
    targets = torch.randint(0, V, (T,), device="cuda", generator=g).int()
    targets[5], targets[8] = 1, 0
    glp, gH = torch.randn(T, device="cuda", generator=g), torch.randn(T, device="cuda", generator=g)
    stats = fp.token_logprobs(logits, targets)["stats"]
    d = fp.token_logprobs_grad(logits, targets, stats, glp, gH)
    sample = torch.tensor([*range(20), T - 1], device="cuda")
    e, tol = grad64(logits[sample], targets[sample], 1.0, glp[sample], gH[sample])
    # the hardware's 2^t is 0 below 2^-126: an e^z up to that, of |z| = 88 and less where it counts most, is left out, and with it
    # p (|g| + |h| |ln p + H|), p <= e^z and |ln p + H| <= |z| + 2 ln V
    lost = 2.0 ** -126 * (glp[sample].abs() + gH[sample].abs() * (88 + 2 * math.log(V)))
    tol = tol + torch.finfo(DT[dtype]).eps / 2 * e.abs() + lost.double().cpu()[:, None]
    assert not bool((~((d[sample].double().cpu() - e).abs() <= tol)).any())
