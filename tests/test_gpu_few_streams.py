"""A FewTokenLayer that is given up while its call on another stream has yet to run: the memory of its
workspace is not handed out before that call is over."""
import pytest

from gpu_util import gpu_ok, print_case, torch
from test_gpu_few import _inputs, _layer

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_ok(), reason="needs a GPU")]


@pytest.mark.parametrize("mode", ["nv", "nvnv", "fp8"])
def test_workspace_outlives_a_call_on_another_stream(mode):
    print_case(f"few given up {mode}")
    import block_scaled_fp4_nvfp4_amd as m
    layer = _layer(mode, 40, 512, 256, 4, seed=7, shared=128)
    x, lg = _inputs(16, 40, 512, seed=8)
    ref = [t.clone() for t in m.FewTokenLayer(layer, 16)(x, lg)]
    out = [torch.zeros_like(t) for t in ref]
    few = m.FewTokenLayer(layer, 16)
    size, at = few.workspace.numel(), few.workspace.data_ptr()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # about 0.1 s: the call is enqueued, not run
        few(x, lg, None, *out)
    del few
    taken = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
    if not side.query():
        assert at not in [t.data_ptr() for t in taken]
    torch.cuda.synchronize()
    for a, b in zip(ref, out):
        assert torch.equal(a, b)
