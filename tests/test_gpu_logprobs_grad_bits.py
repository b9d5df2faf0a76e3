"""token_logprobs_grad keeps its bits where 1 / temperature, the upstream gradients or their quotients by Z are next to the
ends of f32's range, but the result is not (tolerances: test_gpu_logprobs)."""
import pytest

from gpu_util import gpu_ok, print_case, torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_ok(), reason="needs a GPU")]

from head_util import gen  # noqa: E402
from test_gpu_logprobs import DT, _logits, grad64  # noqa: E402


@pytest.mark.parametrize("temperature,size", [(2.0 ** 126, 2.0 ** 60), (1.7e38, 2.0 ** 90), (2.0 ** 120, 2.0 ** 10), (2.0 ** -100, 2.0 ** -120),
                                              (2.0 ** -60, 2.0 ** -126), (1.0, 2.0 ** -60)])
@pytest.mark.parametrize("T,V", [(3, 1001), (2, 20011)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("which", ["logprob", "entropy", "both"])
def test_far_temperatures_and_gradients(temperature, size, T, V, dtype, which):
    """A gradient of the size of d / (T V), every factor of it far from 1.  The last row's logits are all alike, which makes them
    equally likely at any temperature.  (1 / T is one rounding, of a subnormal result above 2^126: 2^-23 more.)"""
    import block_scaled_fp4_nvfp4_amd as fp
    print_case(f"logprobs grad T={T} V={V} {dtype} {which} temperature={temperature} gradients={size}")
    g = gen(V)
    logits = _logits(g, T, V, DT[dtype], pad=5)
    logits[T - 1] = 2.0
    targets = torch.randint(0, V, (T,), device="cuda", generator=g).int()
    glp = (torch.rand(T, device="cuda", generator=g) + 0.5) * size if which != "entropy" else None
    gH = (torch.rand(T, device="cuda", generator=g) - 1.5) * size if which != "logprob" else None
    stats = fp.token_logprobs(logits, targets, temperature=temperature)["stats"]
    d = fp.token_logprobs_grad(logits, targets, stats, glp, gH, temperature)
    e, tol = grad64(logits, targets, temperature, glp, gH)
    tol = tol + (torch.finfo(DT[dtype]).eps / 2 + 2.0 ** -23) * e.abs() + torch.finfo(DT[dtype]).smallest_normal * 2.0 ** -7
    bad = ~((d.double().cpu() - e).abs() <= tol)
    assert not bool(bad.any()), (int(bad.sum()), float(((d.double().cpu() - e).abs() / e.abs().clamp(min=1e-300))[bad].max()))
