"""Arguments of the layer operators that the binding or the C ABI refuses, without a GPU."""
import pytest

torch = pytest.importorskip("torch")

from test_layer_abi import FAKE, Rows, norm, recur  # noqa: E402


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


def test_a_step_in_place_has_the_same_rows(layer):
    """In an input's place a shifted or strided row would be read after it was written.  With
    sizes beyond a launch, so that what is not refused for that is refused for them."""
    L, big = layer._lib(), 1 << 22
    x = Rows(9 * FAKE, 64, 0)
    for name in ("x", "gate", "input_gate"):
        for seqs, seq, want in ((big, 64, 2), (big, 65, 1), (3, 65, 1)):
            c = recur(seqs=seqs, channels=64, **{name: x}, out=Rows(9 * FAKE, seq, 0),
                      **{k: Rows(2 * FAKE, 64, 0) for k in ("x", "gate", "input_gate") if k != name})
            assert L.canon_gated_recurrence_step(c, None) == want, (name, seqs, seq)


def test_norm_eps(layer):
    """Neither negative nor NaN nor infinite; the backward pass does not read it."""
    L, nan, inf = layer._lib(), float("nan"), float("inf")
    for eps in (-1e-5, -inf, nan, inf, 1e39):
        assert L.canon_layer_norm(norm(eps=eps), None) == 1, eps
        assert L.canon_layer_norm_grad(norm(eps=eps), None, 0, None) == 3
    for eps in (0.0, -0.0, 1e-5, 1e38):
        assert L.canon_layer_norm(norm(eps=eps, rows=0), None) == 0, eps
