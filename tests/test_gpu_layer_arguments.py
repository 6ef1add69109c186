"""Arguments at the edge of what the layer operators take."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def canon():
    import scan_canonical_reduce_amd as c
    return c


@pytest.fixture(autouse=True)
def seed():
    torch.manual_seed(5)


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


def test_norm_eps(canon):
    """Any finite eps that is not negative; without one a row of deviations of 2^-60."""
    x, w = torch.randn(5, 300, device="cuda"), torch.ones(300, device="cuda")
    for eps in (-1e-6, float("nan"), float("inf")):
        with pytest.raises(ValueError):
            canon.layer_norm(x, w, eps=eps)
        with pytest.raises(ValueError):
            canon.add_layer_norm(x, x, w, eps=eps)
    for scale in (2.0 ** -60, 1.0, 2.0 ** 60):
        d = (x.double() - x.double().mean(1, keepdim=True)) * scale
        want = d / d.pow(2).mean(1, keepdim=True).sqrt()
        got = canon.layer_norm(x * scale, w, eps=0.0)
        # some 40 roundings of the row's sums and of each value
        assert ((got - want).abs() <= 64 * 2.0 ** -24 * (1 + want.abs())).all()


@pytest.mark.parametrize("width", [60, 700, 4000, 9000, 20001])
def test_norm_of_any_size(canon, width):
    """Rows whose squares leave 32 bits on either side have the outputs of the same rows times
    a power of two, and leave the rows beside them as they are.  The rows' means are their
    sums' rounding, some 2^-26, which times 2^-100 is below the least normal number 2^-126: a
    multiple of 2^-149 there, so each side's may be off by half of that.  A deviation of such a
    row, some 2^-100, has steps of 2^-123, which that does not move."""
    x = torch.randn(24, width, device="cuda")
    x -= x.mean(1, keepdim=True)
    x = torch.where(x.abs() < 2.0 ** -20, 2.0 ** -20, x)  # so that 2^-100 times it is normal
    w, b = torch.rand(width, device="cuda"), torch.rand(width, device="cuda")
    scale = torch.tensor([2.0 ** k for k in (0, -90, 0, 55, 80, -60, 0, 100, -100, 30, -30, 0)] * 2,
                         device="cuda")[:, None]
    stats, own = canon.layer_norm_stats(x), canon.layer_norm_stats(x)
    want = canon.layer_norm(x, w, b, eps=0.0, stats=own)
    out = canon.layer_norm(x * scale, w, b, eps=0.0, stats=stats)
    assert torch.equal(out, want)
    assert ((stats[:, 0].double() - own[:, 0].double() * scale[:, 0]).abs() <= 2.0 ** -149).all()
    assert torch.equal(stats[:, 1], own[:, 1] / scale[:, 0])
    dout = torch.randn_like(x)
    g = canon.layer_norm_grad(dout, x * scale, w, stats, b)
    h = canon.layer_norm_grad(dout, x, w, own, b)
    # of 2^100, where a gradient is not a normal number, rounded to steps of 2^-149 twice
    assert ((g.dx.double() - h.dx.double() / scale).abs() <=
            torch.where((h.dx / scale).abs() < 2.0 ** -126, 2.0 ** -149, 0.0)).all()
    assert torch.equal(g.dweight, h.dweight) and torch.equal(g.dbias, h.dbias)


@pytest.mark.parametrize("decay", [False, True])
def test_sequences_without_rows(canon, decay):
    """States and their gradients pass through; a decay's gradient is zero."""
    x = torch.empty(3, 0, 70, device="cuda")
    init, dfinal = torch.randn(3, 70, device="cuda"), torch.randn(3, 70, device="cuda")
    d = torch.rand(70, device="cuda") if decay else None
    final, keep = torch.zeros_like(init), canon.gated_recurrence_states(x)
    out = canon.gated_recurrence(x, x, d, x, init_state=init, final_state=final, states=keep)
    assert out.shape == x.shape and torch.equal(final, init)
    g = canon.gated_recurrence_grad(x, x, x, keep, d, x, d_final_state=dfinal)
    assert torch.equal(g.dinit_state, dfinal) and g.dx.shape == x.shape
    assert g.ddecay is None if d is None else not g.ddecay.any()
