"""Sums over rows of tensors of more than 2^31 elements: gradients that reach a few rows at
the start, around element 2^31 and at the end alone, so that a row too many or too few
shows."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import layer_ref  # noqa: E402

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module")
def canon():
    import scan_canonical_reduce_amd as c
    yield c
    torch.cuda.empty_cache()


@pytest.fixture(autouse=True)
def seed():
    torch.manual_seed(5)


def normal(*shape, dtype=BF16):
    return torch.empty(*shape, dtype=dtype, device="cuda").normal_()


@pytest.mark.parametrize("rows,width", [(530_000, 4104), (70_000, 32_771)])
def test_norm(canon, rows, width):
    x, w, b = normal(rows, width), normal(width, dtype=F32), normal(width, dtype=F32)
    assert x.numel() > 1 << 31
    stats = canon.layer_norm_stats(x)
    out = canon.layer_norm(x, w, b, stats=stats)
    dout = out.zero_()
    at = (1 << 31) // width
    some = torch.cat([torch.arange(0, 70), torch.arange(at - 70, at + 70),
                      torch.arange(rows - 70, rows)]).cuda()
    dout[some] = normal(len(some), width)
    g = canon.layer_norm_grad(dout, x, w, stats, b)
    mean, rstd = stats[some].to(F64).unbind(1)
    terms = dout[some].to(F64)
    n = (x[some].to(F64) - mean[:, None]) * rstd[:, None]
    # a chunk's 64 rows, its teams, the chunks over 16 lanes and a tree, as many roundings of
    # the absolute sum at most (rows of zeros add none); n's own two
    depth = 64 + 4 + max(512, rows // 64) // 16 + 5
    for got, t, own in ((g.dweight, terms * n, 2), (g.dbias, terms, 0)):
        bound = (depth + own) * layer_ref.U * t.abs().sum(0)
        assert ((got - t.sum(0)).abs() <= bound).all()
        # one row more or less would show in nearly every column
        assert (t.abs().median(0).values > 4 * bound).float().mean() > 0.9


@pytest.mark.parametrize("seqs,rows", [(1, 1 << 21), (512, 1 << 12)])
def test_recurrence(canon, seqs, rows):
    ch, part = 1030, 4096
    x, gate = normal(seqs, rows, ch), normal(seqs, rows, ch)
    assert x.numel() > 1 << 31
    decay = 0.05 + 0.1 * torch.rand(ch, device="cuda")
    states = canon.gated_recurrence_states(x)
    out = canon.gated_recurrence(x, gate, decay, states=states)
    dout = out.zero_()
    # gradients reach back some hundred rows: a is exp(-0.02) at a median
    dout[0, :200], dout[-1, -200:] = normal(200, ch), normal(200, ch)
    g = canon.gated_recurrence_grad(dout, x, gate, states, decay)
    want, size = 0, 0
    for s, t in ((slice(0, 1), slice(0, part)), (slice(seqs - 1, seqs), slice(rows - part, rows))):
        state = torch.zeros(1, ch, device="cuda")
        if t.start:
            canon.gated_recurrence(x[s, :t.start], gate[s, :t.start], decay, final_state=state)
        keep = canon.gated_recurrence_states(x[s, t])
        canon.gated_recurrence(x[s, t], gate[s, t], decay, init_state=state, states=keep)
        h = canon.gated_recurrence_grad(dout[s, t], x[s, t], gate[s, t], keep, decay)
        assert torch.equal(h.dgate, g.dgate[s, t])
        want = want + h.ddecay.to(F64)
        # a gate's gradient is its share of the decay's, times decay (1 - sigmoid(gate))
        share = decay * torch.sigmoid(-gate[s, t].to(F64))
        size = size + (h.dgate.to(F64).abs() / share).sum((0, 1))
    # 64 rows of a wave and the waves of each sum, the blocks over 16 lanes and a tree; the
    # same of the parts'; dgate's own rounding
    blocks = seqs * (rows // 512)
    bound = (2 * (64 + 10) + blocks // 16 + 8) * layer_ref.U * size * (1 + 2.0 ** -7)
    assert ((g.ddecay - want).abs() <= bound).all()
    assert (want.abs() > 4 * bound).float().mean() > 0.9
