"""Sizes of the memory layer's entry points at the edges of the integers that carry them: host
side only, so they run without a GPU."""
import pytest
import torch


@pytest.fixture(scope="module")
def layer():
    import trellis_row_decode_gb300 as cp
    from trellis_row_decode_gb300 import build_ext, layer
    if not cp.LIB_PATH.exists():
        build_ext.build()
    layer._lib()
    return layer


def test_sizes_past_32_bits_are_refused(layer):
    """The ABI's 32-bit sizes: ctypes cuts larger ones, so the binding refuses them."""
    for shape in [(1, 1 << 32), (1 << 32,), (2, 1, (1 << 32) + 8), (0, 1 << 33)]:
        with pytest.raises(ValueError, match=r"2\^32"):
            layer._rows(torch.empty(shape, device="meta"), "x")
    assert layer._rows(torch.empty((3, (1 << 32) - 1), device="meta"), "x") == \
        (3, (1 << 32) - 1, (1 << 32) - 1)
    for call in [lambda: layer.embed_grad_workspace(4, 4, (1 << 32) + 8),
                 lambda: layer.embed_grad_workspace(4, 4, -8),
                 lambda: layer.rms_norm_grad_workspace(4, (1 << 32) + 8),
                 lambda: layer.rms_norm_grad_workspace(4, -8)]:
        with pytest.raises(ValueError, match=r"2\^32"):
            call()
