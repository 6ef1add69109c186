"""Arguments at the edge of what the layer operators take."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def canon():
    import scan_canonical_reduce_amd as c
    return c


def test_a_step_in_place(canon):
    """An output in the place of any input with the same rows; a wider or shifted one is
    refused."""
    for dtype in (torch.float32, torch.bfloat16):
        row = [torch.randn(9, 70, device="cuda").to(dtype) for _ in range(3)]
        decay, state = torch.rand(70, device="cuda"), torch.randn(9, 70, device="cuda")
        want_state = state.clone()
        want = canon.gated_recurrence_step(want_state, row[0], row[1], decay, row[2])
        for i in range(3):
            r, s = [t.clone() for t in row], state.clone()
            got = canon.gated_recurrence_step(s, r[0], r[1], decay, r[2], out=r[i])
            assert got is r[i] and torch.equal(got, want) and torch.equal(s, want_state)
        big = torch.zeros(20, 75, device="cuda", dtype=dtype)
        with pytest.raises(ValueError):
            canon.gated_recurrence_step(state.clone(), big[:9, :70], row[1], decay, row[2],
                                        out=big[:18:2, :70])
