"""A gate that makes a zero ends a sequence in the middle: what follows has the accuracy of
a sequence of its own, whatever size the state had, and gradients do not reach back."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import layer_ref  # noqa: E402

F32, BF16 = torch.float32, torch.bfloat16
BIG = 2.0 ** 40


@pytest.fixture(scope="module")
def canon():
    import scan_canonical_reduce_amd as c
    return c


@pytest.fixture(autouse=True)
def seed():
    torch.manual_seed(5)


def inputs(dtype, n, rows, cut, channels, decay):
    """x before the cut and dout behind it are large; a of row `cut` is 0."""
    g = torch.Generator().manual_seed(rows + cut)
    x, gate, dout = (torch.randn(n, rows, channels, generator=g) for _ in range(3))
    x[:, :cut] *= BIG
    dout[:, cut:] *= BIG
    if decay:
        d = 200 + torch.rand(channels, generator=g)  # exp(-200) is 0 in 32 bits
        gate -= 8
        gate[:, cut] = 40.0
    else:
        d = None
        gate += 2
        gate[:, cut] = -float("inf")
    init = BIG * torch.randn(n, channels, generator=g)
    return [None if t is None else t.cuda() for t in
            (x.to(dtype), gate.to(dtype), dout.to(dtype), d, init)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("decay", [False, True])
@pytest.mark.parametrize("n,rows,channels,cuts", [
    (2, 300, 66, (1, 3, 8, 121, 127, 128, 200)),         # a workgroup for each round
    (1, 1500, 66, (5, 512, 515, 640, 1023, 1400)),       # the same, of several blocks
    (70, 200, 70, (64, 131)),                            # for each block
    (3, 1100, 3000, (300, 1024, 1027)),                  # for each block, two channels a lane
    (260, 1100, 20, (100, 700, 1030)),                   # whole sequences
    (1, 17 * 1024, 8, (17, 9000, 17000))])               # more blocks than each folds
def test_after_a_reset(canon, dtype, decay, n, rows, channels, cuts):
    for cut in cuts:
        x, gate, dout, d, init = inputs(dtype, n, rows, cut, channels, decay)
        states = canon.gated_recurrence_states(x)
        final = torch.empty_like(init)
        out = canon.gated_recurrence(x, gate, d, init_state=init, final_state=final, states=states)
        g = canon.gated_recurrence_grad(dout, x, gate, states, d)
        some = slice(0, min(n, 4))  # the sequences compared
        end = min(rows, cut + 300)
        after = layer_ref.recur(x[some, cut:end], gate[some, cut:end].clamp(min=-80), None, d)
        layer_ref.within(out[some, cut:end], *after["out"], f"out, cut {cut}")
        if end == rows:
            layer_ref.within(final[some], *after["final"], f"final, cut {cut}")
        first = max(0, cut - 300)
        before = layer_ref.recur(x[some, first:cut], gate[some, first:cut], None, d,
                                 dout=dout[some, first:cut])
        layer_ref.within(g.dx[some, first:cut], *before["x"], f"dx, cut {cut}")
        if first == 0:
            layer_ref.within(g.dinit_state[some], *before["init"], f"dinit, cut {cut}")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_step(canon, dtype):
    state = torch.full((5, 130), BIG, device="cuda")
    x = torch.randn(5, 130, device="cuda").to(dtype)
    gate = torch.full_like(x, -float("inf"))
    assert torch.equal(canon.gated_recurrence_step(state, x, gate), x)
    assert torch.equal(state, x.float())


def test_packed(canon):
    """Resets as ends of sequences: the outputs of the sequences packed."""
    lens = [5, 64, 1, 130, 700, 13]
    ends = [0]
    for n in lens:
        ends.append(ends[-1] + n)
    g = torch.Generator().manual_seed(5)
    x, gate = (torch.randn(ends[-1], 70, generator=g).cuda() for _ in range(2))
    gate = gate + 2
    gate[ends[:-1]] = -float("inf")
    x[ends[1]:ends[2]] *= BIG
    one = canon.gated_recurrence(x[None], gate[None])[0]
    for a, b in zip(ends, ends[1:]):
        r = layer_ref.recur(x[None, a:b], gate[None, a:b].clamp(min=-80))
        layer_ref.within(one[None, a:b], *r["out"], f"rows {a} to {b}")


@pytest.mark.parametrize("n,rows,channels", [(1, 512, 66), (2, 1500, 66), (70, 512, 70),
                                             (260, 1100, 20)])
def test_a_slow_loss_is_not_rounded_away(canon, n, rows, channels):
    """An a of 1 - 2^-28 over many rows of no input: a chunk of 8 rows takes less than half
    of the state's last bit, which chunk by chunk in 32 bits would all be lost, 7 of these
    roundings U within a round.  An output is off by the rounding of its chunk's start, U / 2,
    and by up to 8 rows' loss, 0.48 U.  Gradients of x are the state's, times a constant: two
    roundings more of each of the two that are compared."""
    x = torch.zeros(n, rows, channels, device="cuda")
    gate = torch.full_like(x, 19.45)
    ones = torch.ones(n, channels, device="cuda")
    states = canon.gated_recurrence_states(x)
    out = canon.gated_recurrence(x, gate, init_state=ones, states=states)
    e = torch.sigmoid(-gate[0, 0, 0].double())
    t = torch.arange(1, rows + 1, device="cuda", dtype=torch.float64)
    want = torch.exp(t * torch.log1p(-e))[:, None]
    assert ((out - want).abs() <= 1.25 * layer_ref.U).all()
    g = canon.gated_recurrence_grad(x, x, gate, states, d_final_state=ones)
    ratio = g.dx.double() / g.dx[:, -1:].double()
    assert ((ratio - want.flip(0) / want[0]).abs() <= 4 * layer_ref.U).all()
