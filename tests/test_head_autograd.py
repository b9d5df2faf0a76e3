"""Operands that require a gradient: a result without a graph would leave its gradient out of a training step silently, so the
calls refuse them while gradients are enabled, and are used from a torch.autograd.Function."""
import pytest

torch = pytest.importorskip("torch")

from gpu_util import gpu_ok  # noqa: E402


def _record(device="cpu", n=32, k=64):
    return {"codes": torch.full((n, k // 2), 0x2A, dtype=torch.uint8, device=device),
            "scales": torch.full((n, k // 16), 0x38, dtype=torch.uint8, device=device), "tensor_scale": torch.ones(1, device=device)}


def test_refused_while_gradients_are_enabled():
    import block_scaled_fp4_nvfp4_amd as fp
    x, dy, plain = torch.zeros(3, 64, requires_grad=True), torch.zeros(3, 32, requires_grad=True), torch.zeros(3, 64)
    for call in (lambda: fp.fp4_matmul(x, _record(), "nvfp4"), lambda: fp.fp4_matmul_grad(dy, _record(), "nvfp4"),
                 lambda: fp.fp4_matmul(plain, {**_record(), "tensor_scale": torch.ones(1, requires_grad=True)}, "nvfp4"),
                 lambda: fp.fp4_matmul(plain, _record(), "nvfp4", out_dtype=torch.float32, out=torch.zeros(3, 32, requires_grad=True)),
                 lambda: fp.token_logprobs(x, None), lambda: fp.token_logprobs_grad(x, None, torch.zeros(3, 3), None),
                 lambda: fp.token_logprobs_grad(plain, None, torch.zeros(3, 3), None, torch.zeros(3, requires_grad=True)),
                 lambda: fp.token_logprobs_grad(plain, None, torch.zeros(3, 3), None, out=x)):
        with pytest.raises(ValueError, match="requires a gradient"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="device tensor"):  # host tensors: the next check
            call()


@pytest.mark.gpu
@pytest.mark.skipif(not gpu_ok(), reason="needs a GPU")
def test_in_an_autograd_function():
    """The calls as forward and backward of functions, under a sum that uses x on another way too, against float64's autograd.
    Exact operands and few bits: logits are exact.  The logits' gradient moves by f32's rounding of p, ln Z and H, 400 u (1 +
    max |ln p|) times the upstream gradients at most (as in the training step of the head's tests), times sum |W| for x's; x's two
    parts are added with a rounding each."""
    import block_scaled_fp4_nvfp4_amd as fp

    class Product(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w):
            ctx.w = w
            return fp.fp4_matmul(x, w, "nvfp4", out_dtype=torch.float32)

        @staticmethod
        def backward(ctx, dy):
            return fp.fp4_matmul_grad(dy.contiguous(), ctx.w, "nvfp4", out_dtype=torch.float32), None

    class Logprob(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, targets):
            r = fp.token_logprobs(logits, targets)
            ctx.save_for_backward(logits, targets, r["stats"])
            return r["logprobs"], r["entropy"].clone()

        @staticmethod
        def backward(ctx, d_logprobs, d_entropy):
            logits, targets, stats = ctx.saved_tensors
            return fp.token_logprobs_grad(logits, targets, stats, d_logprobs.contiguous(), d_entropy.contiguous()), None

    g = torch.Generator(device="cuda").manual_seed(1)
    w = _record("cuda")
    w["codes"] = torch.randint(0, 256, w["codes"].shape, dtype=torch.uint8, device="cuda", generator=g)
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device="cuda")
    W = torch.stack((grid[w["codes"].int() & 15], grid[w["codes"].int() >> 4]), -1).flatten(-2)
    x = torch.randint(-2, 3, (5, 64), device="cuda", generator=g).float() / 16
    targets = torch.randint(0, 32, (5,), device="cuda", generator=g).int()

    def loss(x, logits, chosen, H):
        return chosen.sum() - 0.25 * H.sum() + (x * x).sum()

    a = x.clone().requires_grad_()
    logits = Product.apply(a, w)
    loss(a, logits, *Logprob.apply(logits, targets)).backward()
    b = x.double().requires_grad_()
    lp = torch.log_softmax(b @ W.t().contiguous(), 1)
    loss(b, None, lp.gather(1, targets[:, None].long())[:, 0], -(lp.exp() * lp).sum(1)).backward()
    assert torch.equal(logits.detach().double(), x.double() @ W.t().contiguous())
    most = lp.detach().abs().max()
    move = (1 + 0.25 * (2 + most)) * 400 * 2.0 ** -24 * (1 + most)
    assert bool(((a.grad.double() - b.grad).abs() <= move * W.abs().sum(0) + 2.0 ** -22 * (b.grad.abs() + 2 * b.detach().abs())).all())
