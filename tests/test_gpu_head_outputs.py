"""The results of fp4_matmul, fp4_matmul_grad, token_logprobs and token_logprobs_grad are allocated where torch can see it: by
its dispatch modes, its deterministic mode, and in spite of a change of its short way to memory."""
import pytest

from gpu_util import gpu_ok, print_case, torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_ok(), reason="needs a GPU")]

from head_util import gen, raw_weight  # noqa: E402


def _all(x, dy, w, logits, targets):
    """Every tensor that the four calls return."""
    import block_scaled_fp4_nvfp4_amd as fp
    r = fp.token_logprobs(logits, targets, top=3)
    ones = torch.ones(len(targets), device="cuda")
    return [fp.fp4_matmul(x, w, "nvfp4"), fp.fp4_matmul_grad(dy, w, "nvfp4"), *r.values(),
            fp.token_logprobs_grad(logits, targets, r["stats"], ones)]


@pytest.fixture
def operands():
    g = gen(5)
    return (torch.randn(1, 5, 64, device="cuda", generator=g), torch.randn(1, 5, 48, device="cuda", generator=g), raw_weight(g, "nvfp4", 1, 48, 64),
            torch.randn(4, 3000, device="cuda", generator=g), torch.tensor([0, 5, -1, 2999], dtype=torch.int32, device="cuda"))


def test_a_dispatch_mode_sees_the_results(operands):
    from torch.utils._python_dispatch import TorchDispatchMode
    print_case("dispatch mode")

    class Seen(TorchDispatchMode):
        def __init__(self):
            super().__init__()
            self.memory = set()

        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            out = func(*args, **(kwargs or {}))
            if isinstance(out, torch.Tensor):
                self.memory.add(out.untyped_storage().data_ptr())
            return out

    want = _all(*operands)
    with Seen() as seen:
        got = _all(*operands)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(t.untyped_storage().data_ptr() in seen.memory for t in got)


def test_deterministic_mode_and_another_signature(operands, monkeypatch):
    from block_scaled_fp4_nvfp4_amd import _lib
    print_case("deterministic mode, other signature")
    want = _all(*operands)
    calls = []
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: (calls.append(a), empty(*a, **k))[1])
    torch.use_deterministic_algorithms(True, warn_only=True)
    try:
        got = _all(*operands)
    finally:
        torch.use_deterministic_algorithms(False)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and len(calls) >= 8
    del calls[:]

    def other(*args):
        raise TypeError("other arguments expected")
    monkeypatch.setattr(_lib, "_empty_strided_cuda", other)
    got = _all(*operands)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and len(calls) >= 8
