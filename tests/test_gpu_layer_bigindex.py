"""The layer operators on tensors of more than 2^31 elements: the rows at the end have
the bits they have alone."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def canon():
    import scan_canonical_reduce_amd as c
    yield c
    torch.cuda.empty_cache()


def normal(*shape, dtype=BF16):
    return torch.empty(*shape, dtype=dtype, device="cuda").normal_()


def test_norm(canon):
    x, r = normal(530_000, 4104), normal(530_000, 4104)
    w, b = normal(4104, dtype=torch.float32), normal(4104, dtype=torch.float32)
    assert x.numel() > 1 << 31
    stats = canon.layer_norm_stats(x)
    out, total = canon.add_layer_norm(x, r, w, b, stats=stats)
    tail = slice(-70, None)
    own = canon.layer_norm_stats(x[tail])
    one, one_total = canon.add_layer_norm(x[tail], r[tail], w, b, stats=own)
    assert torch.equal(out[tail], one) and torch.equal(total[tail], one_total)
    assert torch.equal(stats[tail], own)
    g = canon.layer_norm_grad(r, total, w, stats, b, dsum=x, dx=out)
    h = canon.layer_norm_grad(r[tail], one_total, w, own, b, dsum=x[tail])
    assert torch.equal(g.dx[tail], h.dx)


def test_very_wide_norm(canon):
    x = normal(70_000, 32_771)
    w = normal(32_771, dtype=torch.float32)
    assert x.numel() > 1 << 31
    stats = canon.layer_norm_stats(x)
    out = canon.layer_norm(x, w, stats=stats)
    tail = slice(-9, None)
    own = canon.layer_norm_stats(x[tail])
    assert torch.equal(out[tail], canon.layer_norm(x[tail], w, stats=own))
    g = canon.layer_norm_grad(out, x, w, stats)
    assert torch.equal(g.dx[tail], canon.layer_norm_grad(out[tail], x[tail], w, own).dx)


@pytest.mark.parametrize("seqs,rows", [(1, 1 << 21), (512, 1 << 12)])
def test_recurrence(canon, seqs, rows):
    """One sequence in blocks, many whole; the last 1000 rows and some again from the
    state before them."""
    ch = 1030
    x, gate, dout = (normal(seqs, rows, ch) for _ in range(3))
    assert x.numel() > 1 << 31
    decay = torch.rand(ch, device="cuda") * 0.1
    states = canon.gated_recurrence_states(x)
    final = torch.empty(seqs, ch, device="cuda")
    out = canon.gated_recurrence(x, gate, decay, None, final_state=final, states=states)
    g = canon.gated_recurrence_grad(dout, x, gate, states, decay)
    cut, s = rows - 2 * 512, slice(seqs - 1, seqs)
    state = torch.empty(1, ch, device="cuda")
    canon.gated_recurrence(x[s, :cut], gate[s, :cut], decay, final_state=state)
    xt, gt = x[s, cut:], gate[s, cut:]
    keep = canon.gated_recurrence_states(xt)
    tail = canon.gated_recurrence(xt, gt, decay, None, None, state, state, keep)
    assert torch.equal(tail, out[s, cut:]) and torch.equal(state, final[s])
    h = canon.gated_recurrence_grad(dout[s, cut:], xt, gt, keep, decay)
    assert torch.equal(h.dx, g.dx[s, cut:]) and torch.equal(h.dgate, g.dgate[s, cut:])


def test_sampling(canon):
    x = normal(17_000, 131_075, dtype=torch.float16)
    assert x.numel() > 1 << 31
    u = torch.rand(17_000, device="cuda")
    for kw in ({}, dict(top_k=40), dict(top_p=0.8)):
        got = canon.sample(x, u, **kw)
        assert torch.equal(got[-40:], canon.sample(x[-40:], u[-40:], **kw))
