"""examples/memory_layer.py: the memory layer's operators as they are used together."""
import importlib.util
from pathlib import Path

import pytest

pytestmark = pytest.mark.gpu


def test_memory_layer_trains_compresses_and_serves():
    path = Path(__file__).resolve().parent.parent / "examples" / "memory_layer.py"
    spec = importlib.util.spec_from_file_location("memory_layer_example", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses, off, off_one = m.main()
    assert losses[-1] < 0.9 * losses[0]
    # 2-bit codes of Gaussian rows are off by less than sqrt(0.1175) (the best scalar 4-level
    # quantiser's distortion) of the memory's share; e4m3 adds under 2^-4
    assert off < 0.1175 ** 0.5 + 2.0 ** -4
    assert off_one < 1.5 * (0.1175 ** 0.5 + 2.0 ** -4)
