"""moe_fp4_forward_few refuses bad arguments on the host (no GPU needed:
every call here returns before any HIP call)."""
import ctypes

import pytest

pytest.importorskip("torch")


@pytest.fixture(scope="module")
def L():
    from block_scaled_fp4_nvfp4_amd import _lib
    return _lib.lib()


FAKE = ctypes.c_void_p(0x1000)


def _layer(**kw):
    from block_scaled_fp4_nvfp4_amd import _lib
    s = _lib.LayerStruct()
    base = dict(w_fmt=0, a_fmt=5, num_experts=8, hidden=256, inter=128, top_k=2)
    base.update({k: 0x1000 for k in ("w13", "w13_scale", "w13_scale_2", "w2", "w2_scale", "w2_scale_2")})
    base.update(kw)
    for k, v in base.items():
        setattr(s, k, v)
    return s


def _size(L, s, t):
    n = ctypes.c_size_t()
    return L.moe_fp4_few_workspace_size(ctypes.byref(s), t, ctypes.byref(n)), n.value


def _call(L, s, t=2, x=FAKE, lg=FAKE, bias=None, y=FAKE, yd=1, ids=None, w=None, ws=FAKE, wb=1 << 30):
    return L.moe_fp4_forward_few(ctypes.byref(s), x, t, lg, bias, y, yd, ids, w, ws, wb, None)


def test_layer_refusals(L):
    assert _size(L, _layer(), 1)[0] == 0 and _size(L, _layer(), 16)[0] == 0
    assert _size(L, _layer(), 17)[0] == -3                                   # few tokens only
    assert _size(L, _layer(), -1)[0] == -2
    assert _size(L, _layer(num_experts=1025), 1)[0] == -3
    assert _size(L, _layer(top_k=9), 1)[0] == -1 and _size(L, _layer(top_k=0), 1)[0] == -1
    assert _size(L, _layer(num_experts=64, top_k=33), 1)[0] == -1
    assert _size(L, _layer(hidden=250), 1)[0] == -2
    assert _size(L, _layer(w_fmt=0, a_fmt=2), 1)[0] == -3                    # format pair
    assert _size(L, _layer(hidden=96, inter=96), 1)[0] == 0
    assert _size(L, _layer(hidden=96, inter=96, shared_inter=128), 1)[0] == -2
    assert _size(L, _layer(hidden=4096), 8)[0] == 0 and _size(L, _layer(hidden=8192), 16)[0] == -3  # LDS
    assert _size(L, _layer(a_fmt=0, hidden=32768, inter=65536), 1)[0] == 0
    assert _size(L, _layer(a_fmt=0, hidden=65536, inter=65536), 1)[0] == -3  # an expert's rows exceed a buffer descriptor
    assert _size(L, _layer(hidden=256, inter=65536), 1)[0] == -3             # two terms of h exceed the LDS
    assert L.moe_fp4_few_workspace_size(ctypes.byref(_layer()), 1, None) == -1
    assert L.moe_fp4_few_workspace_size(None, 1, ctypes.byref(ctypes.c_size_t())) == -1
    sizes = [_size(L, _layer(), t)[1] for t in range(1, 17)]
    assert sizes == sorted(sizes)                                            # a workspace for 16 serves fewer


def test_call_refusals(L):
    s = _layer()
    odd = ctypes.c_void_p(0x1008)
    assert _call(L, s, yd=2) == -1
    for kw in ("x", "lg", "y"):
        assert _call(L, s, **{kw: None}) == -1, kw
    assert _call(L, s, x=odd) == -1 and _call(L, s, y=ctypes.c_void_p(0x1002)) == -1
    assert _call(L, s, bias=ctypes.c_void_p(0x1001)) == -1 and _call(L, s, ids=ctypes.c_void_p(0x1002)) == -1
    assert _call(L, s, ws=None) == -4 and _call(L, s, wb=_size(L, s, 2)[1] - 1) == -4
    assert _call(L, s, ws=odd) == -1
    assert _call(L, _layer(w13=None)) == -1 and _call(L, _layer(w2_scale_2=None)) == -1
    assert _call(L, _layer(w13=0x1008)) == -1 and _call(L, _layer(w13_scale=0x1001)) == -1
    assert _call(L, _layer(w_fmt=3, a_fmt=4, w2_scale=0x1002)) == -1
    assert _call(L, _layer(shared_inter=128)) == -1                          # shared tensors missing
    assert _call(L, s, t=17) == -3
    assert _call(L, s, t=0, x=None, lg=None, y=None, ws=None, wb=0) == 0     # nothing to do


def test_binding_refusals():
    import torch

    import block_scaled_fp4_nvfp4_amd as fp
    z = torch.zeros(8, 4, dtype=torch.uint8)
    layer = fp.MoELayer("nvfp4", "none", 8, 256, 128, 2, z, z, z, z, z, z)
    with pytest.raises(TypeError):
        fp.FewTokenLayer(layer, 4, torch.float16)
    with pytest.raises(fp.Fp4Error):
        fp.FewTokenLayer(layer, 17)
    few = fp.FewTokenLayer(layer, 4)
    x, lg = torch.zeros(2, 256, dtype=torch.bfloat16), torch.zeros(2, 8)
    for bad in (dict(x=x.float()), dict(x=x[:, :128]), dict(x=torch.zeros(5, 256, dtype=torch.bfloat16)), dict(logits=lg[:1]),
                dict(logits=lg.double()), dict(logits=torch.zeros(8, 2).t()), dict(bias=torch.zeros(7)),
                dict(y=torch.zeros(2, 256, dtype=torch.bfloat16)), dict(topk_ids=torch.zeros(2, 2)),
                dict(topk_weights=torch.zeros(2, 3))):
        with pytest.raises(ValueError):
            few(**{"x": x, "logits": lg, **bad})
