"""Arguments of the layer operators that the binding or the C ABI refuses, without a GPU."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def layer():
    from scan_canonical_reduce_amd import layer as m
    return m


def test_top_k_is_an_integer(layer):
    import numpy as np
    for v in (50.0, 0.5, "3", None):
        with pytest.raises(TypeError, match="top_k must be an integer"):
            layer._setting("sample", "top_k", v, 3, torch.int32)
    for v in (50, np.int64(50), np.int32(50)):
        assert layer._setting("sample", "top_k", v, 3, torch.int32) == (0, 50)
    assert layer._setting("sample", "top_p", 0.5, 3, torch.float32) == (0, 0.5)
