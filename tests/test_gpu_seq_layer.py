"""The operators as a sequence layer uses them together: embedding, causal
convolution, selective scan and back; streams, graphs, decoding."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import seq_ref  # noqa: E402

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def canon():
    import scan_canonical_reduce_amd as c
    return c


def layer(dtype=F32, seqs=3, rows=70, vocab=50, width=64, states=16, seed=0):
    g = torch.Generator().manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, generator=g)

    return {k: v.cuda() for k, v in dict(
        ids=torch.randint(0, vocab, (seqs, rows), generator=g), table=normal(vocab, width).to(dtype),
        w=normal(width, 4), b=normal(width), A=-torch.exp(normal(width, states)),
        D=normal(width), delta=normal(seqs, rows, width).to(dtype) - 2,
        B=normal(seqs, rows, states).to(dtype), C=normal(seqs, rows, states).to(dtype),
        z=normal(seqs, rows, width).to(dtype), dout=normal(seqs, rows, width).to(dtype)).items()}


def forward(canon, p):
    x = canon.embedding(p["table"], p["ids"])
    u = canon.causal_conv(x, p["w"], p["b"], "silu")
    keep = canon.selective_scan_states(u, p["A"].shape[1])
    y = canon.selective_scan(u, p["delta"], p["A"], p["B"], p["C"], D=p["D"], z=p["z"],
                             delta_softplus=True, states=keep)
    return x, u, keep, y


def backward(canon, p, x, u, keep):
    s = canon.selective_scan_grad(p["dout"], u, p["delta"], p["A"], p["B"], p["C"], keep,
                                  D=p["D"], z=p["z"], delta_softplus=True)
    c = canon.causal_conv_grad(s.du, x, p["w"], p["b"], "silu")
    e = canon.embedding_grad(c.dx, p["ids"], p["table"].shape[0], dtype=F32)
    return [e, c.dweight, c.dbias, s.dA, s.dD, s.ddelta, s.dB, s.dC, s.dz]


def test_training_step(canon):
    """Loss and every gradient against autograd of the float64 form: float32
    throughout, sums of a few hundred terms, three operators deep.  The bound
    is relative to each tensor's largest value: (5 rows + 64) roundings for the
    scan, twice that backward, as its own tests derive, times the 2^4 by which
    absolute sums of such inputs exceed the values."""
    p = layer()
    x, u, keep, y = forward(canon, p)
    got = backward(canon, p, x, u, keep)
    e = {k: v.double().cpu() if v.is_floating_point() else v.cpu() for k, v in p.items()}
    names = ["table", "w", "b", "A", "D", "delta", "B", "C", "z"]
    for k in names:
        e[k].requires_grad_()
    outs = []
    for i in range(3):
        xi = e["table"][e["ids"][i]]
        ui, _ = seq_ref.conv_one(xi, e["w"], e["b"], True, torch.zeros(3, 64).double())
        outs.append(seq_ref.scan_one(ui, e["delta"][i], e["A"], e["B"][i][:, None],
                                     e["C"][i][:, None], e["D"], e["z"][i], None, True,
                                     torch.zeros(64, 16).double())[0])
    out = torch.stack(outs)
    want = torch.autograd.grad((out * e["dout"]).sum(), [e[k] for k in names])
    bound = 16 * 2 * (5 * 70 + 64) * seq_ref.U32
    for name, a, b in zip(["y"] + names, [y] + got, [out.detach()] + list(want)):
        err = float((a.double().cpu() - b).abs().max() / b.abs().max())
        assert err <= bound, (name, err, bound)


def test_decoding_continues_the_prompt(canon):
    """A prompt, then single rows: the convolution's bits are the sequence's;
    the scan's rows lie within its bound."""
    p = layer(BF16)
    _, u, _, y = forward(canon, p)
    n = 64
    conv = torch.empty(3, 3, 64, dtype=BF16, device="cuda")
    state = torch.empty(3, 64, 16, device="cuda")
    x = canon.embedding(p["table"], p["ids"][:, :n].contiguous())
    un = canon.causal_conv(x, p["w"], p["b"], "silu", final_state=conv)
    assert torch.equal(un, u[:, :n])
    yn = canon.selective_scan(un, p["delta"][:, :n], p["A"], p["B"][:, :n], p["C"][:, :n],
                              D=p["D"], z=p["z"][:, :n], delta_softplus=True, final_state=state)
    assert torch.equal(yn, y[:, :n])
    for t in range(n, 70):
        xt = canon.embedding(p["table"], p["ids"][:, t].contiguous())
        ut = canon.causal_conv_step(xt, conv, p["w"], p["b"], "silu")
        assert torch.equal(ut, u[:, t])
        yt = canon.selective_scan_step(state, ut, p["delta"][:, t], p["A"], p["B"][:, t],
                                       p["C"][:, t], D=p["D"], z=p["z"][:, t],
                                       delta_softplus=True)
        # both are roundings to bfloat16 of values a few float32 roundings apart
        diff = (yt.float() - y[:, t].float()).abs()
        assert (diff <= 2 ** -7 * y[:, t].float().abs() + 1e-4).all()


def test_two_streams(canon):
    """Independent calls on two streams, each with its own buffers."""
    ps = [layer(BF16, rows=300, width=256, seed=s) for s in (1, 2)]
    want = []
    for p in ps:
        x, u, keep, y = forward(canon, p)
        want.append([y] + backward(canon, p, x, u, keep))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    got = [None, None]
    for _ in range(3):
        for i, p in enumerate(ps):
            streams[i].wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(streams[i]):
                x, u, keep, y = forward(canon, p)
                got[i] = [y] + backward(canon, p, x, u, keep)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_graph_capture(canon):
    """The whole step captured, replayed on changed inputs with eager work and
    synchronisations between the replays."""
    p = layer(BF16, rows=130, width=128, seed=3)
    x, u, keep, y = forward(canon, p)
    backward(canon, p, x, u, keep)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x, u, keep, y = forward(canon, p)
        got = [y] + backward(canon, p, x, u, keep)
    for seed in range(4):
        q = layer(BF16, rows=130, width=128, seed=10 + seed)
        for k in p:
            p[k].copy_(q[k])
        graph.replay()
        torch.cuda.synchronize()
        xe, ue, ke, ye = forward(canon, q)
        want = [ye] + backward(canon, q, xe, ue, ke)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), seed


def test_same_bits_every_run(canon):
    p = layer(BF16, seqs=4, rows=257, width=320, seed=4)
    x, u, keep, y = forward(canon, p)
    want = [y] + backward(canon, p, x, u, keep)
    for _ in range(3):
        x, u, keep, y = forward(canon, p)
        got = [y] + backward(canon, p, x, u, keep)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("rows", [0, 5, 64, 300])
def test_rows_of_no_sequence(canon, rows):
    """starts of one value: no sequence, so the parameters' gradients are zero and
    no row is written."""
    starts = torch.tensor([2], dtype=torch.int32, device="cuda")
    x = torch.randn(rows, 40, device="cuda")
    w, b = torch.randn(40, 4, device="cuda"), torch.randn(40, device="cuda")
    out = torch.full_like(x, 7.0)
    canon.causal_conv(x, w, b, "silu", starts, out=out)
    assert (out == 7).all()
    g = canon.causal_conv_grad(x, x, w, b, "silu", starts, dx=out)
    assert (out == 7).all() and not g.dweight.any() and not g.dbias.any()
    A, B, D = -torch.rand(40, 8, device="cuda"), torch.randn(rows, 8, device="cuda"), b
    keep = canon.selective_scan_states(x, 8, starts)
    canon.selective_scan(x, x, A, B, B, D, x, b, True, starts, states=keep, out=out)
    assert (out == 7).all()
    g = canon.selective_scan_grad(x, x, x, A, B, B, keep, D, x, b, True, starts)
    assert not g.dA.any() and not g.dD.any() and not g.ddelta_bias.any()
    assert g.dinit_state.shape == (0, 40, 8)
