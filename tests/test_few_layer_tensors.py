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
