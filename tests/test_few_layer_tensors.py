"""FewTokenLayer keeps what its argument record points at (no GPU needed)."""
import dataclasses
import gc
import weakref

import pytest

torch = pytest.importorskip("torch")


def _layer():
    import block_scaled_fp4_nvfp4_amd as fp
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    E, H, I, S = 4, 256, 128, 128
    return fp.MoELayer("nvfp4", "nvfp4", E, H, I, 2, u8(E, 2 * I, H // 2), u8(E, 2 * I, H // 16), u8(E, H, I // 2), u8(E, H, I // 16),
                       torch.ones(E), torch.ones(E), torch.ones(1), torch.ones(1), S, u8(2 * S, H), u8(2 * S, H // 32),
                       u8(H, S), u8(H, S // 32), torch.zeros(H, dtype=torch.bfloat16))


def test_replaced_tensors_of_the_layer_stay_alive():
    import block_scaled_fp4_nvfp4_amd as fp
    layer = _layer()
    few = fp.FewTokenLayer(layer, 4)
    names = [f.name for f in dataclasses.fields(layer) if isinstance(getattr(layer, f.name), torch.Tensor)]
    assert len(names) == 13
    for name in names:
        held, at = weakref.ref(getattr(layer, name)), getattr(layer, name).data_ptr()
        setattr(layer, name, torch.zeros(1))
        gc.collect()
        assert held() is not None and held().data_ptr() == at, name
        assert at == getattr(few._struct, name), name
    layer.top_k = 3  # sizes are those at construction too
    assert few._struct.top_k == few.layer.top_k == 2


def test_layer_that_is_given_up():
    import block_scaled_fp4_nvfp4_amd as fp
    layer = _layer()
    held = weakref.ref(layer.w13)
    few = fp.FewTokenLayer(layer, 4)
    del layer
    gc.collect()
    assert held() is not None and few.layer.w13 is held()
    del few
    gc.collect()
    assert held() is None


@pytest.mark.parametrize("pair", [("nvfp4", "nvfp4"), ("mxfp4", "mxfp8"), ("fp8_block", "fp8_row")])
def test_tensors_that_the_kernels_could_not_read(pair):
    """Each tensor too small, not contiguous, of another type or on another device: refused before the
    library is called, with its name; as is a whole layer that is not on a GPU."""
    import block_scaled_fp4_nvfp4_amd as fp
    layer = dataclasses.replace(_layer(), w_fmt=pair[0], a_fmt=pair[1])
    E, H, I = layer.num_experts, layer.hidden, layer.inter
    if pair[0] == "fp8_block":
        u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)
        layer = dataclasses.replace(layer, w13=u8(E, 2 * I, H), w13_scale=torch.ones(E, 2 * I // 128, H // 128), w2=u8(E, H, I),
                                    w2_scale=torch.ones(E, H // 128, I // 128))
    if pair[0] == "mxfp4":
        layer = dataclasses.replace(layer, w13_scale=layer.w13_scale[..., : H // 32].contiguous(),
                                    w2_scale=layer.w2_scale[..., : I // 32].contiguous())
    if pair[0] != "nvfp4":
        layer = dataclasses.replace(layer, w13_scale_2=None, w2_scale_2=None, input_scale=None, inter_scale=None)
    x, lg = torch.zeros(2, H, dtype=torch.bfloat16), torch.zeros(2, E)

    def refused(l, match):
        few = fp.FewTokenLayer(l, 2)
        with pytest.raises(ValueError, match=match):
            few(x, lg)

    refused(layer, "device tensors expected")
    for f in dataclasses.fields(layer):
        t = getattr(layer, f.name)
        if not isinstance(t, torch.Tensor):
            continue
        bad = [t.flatten()[:-1], t.double()]
        if t.numel() > 1:
            bad.append(torch.stack((t, t), -1)[..., 0])
        if f.name != "w13":
            bad.append(t.to("meta"))
        for b in bad:
            refused(dataclasses.replace(layer, **{f.name: b}), f.name + ":")
    refused(dataclasses.replace(layer, w13=layer.w13.to("meta")), "on meta expected")
