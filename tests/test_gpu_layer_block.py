"""The layer operators as a recurrent language model uses them together: embedding,
residual blocks of layer norm, convolution and gated recurrence, the next token; a
training step, prompts and single rows, streams, graphs."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import layer_ref  # noqa: E402
import seq_ref  # noqa: E402

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
EPS = 1e-5


@pytest.fixture(scope="module")
def canon():
    import scan_canonical_reduce_amd as c
    return c


def model(dtype=F32, seqs=3, rows=70, vocab=50, width=64, seed=0):
    """One residual block between two norms; the head is the table."""
    g = torch.Generator().manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, generator=g)

    p = dict(ids=torch.randint(0, vocab, (seqs, rows), generator=g),
             table=normal(vocab, width).to(dtype), n1=1 + 0.1 * normal(width),
             b1=0.1 * normal(width), conv=normal(width, 4), cb=normal(width),
             Wg=(normal(width, width) / width ** 0.5).to(dtype),
             Wi=(normal(width, width) / width ** 0.5).to(dtype),
             decay=torch.rand(width, generator=g) * 0.2, n2=1 + 0.1 * normal(width),
             b2=0.1 * normal(width), dout=normal(seqs, rows, width).to(dtype))
    return {k: v.cuda() for k, v in p.items()}


def forward(canon, p, conv=None, state=None, starts=None):
    """conv, state: of the sequences, continued in place where given."""
    s = dict(x=canon.embedding(p["table"], p["ids"]))
    s["st1"], s["st2"] = canon.layer_norm_stats(s["x"]), canon.layer_norm_stats(s["x"])
    s["a"] = canon.layer_norm(s["x"], p["n1"], p["b1"], EPS, stats=s["st1"])
    s["u"] = canon.causal_conv(s["a"], p["conv"], p["cb"], "silu", starts, final_state=conv)
    s["g"], s["i"] = s["a"] @ p["Wg"], s["a"] @ p["Wi"]
    s["keep"] = canon.gated_recurrence_states(s["u"], starts)
    s["h"] = canon.gated_recurrence(s["u"], s["g"], p["decay"], s["i"], starts, None, state,
                                    s["keep"])
    s["y"], s["sum"] = canon.add_layer_norm(s["h"], s["x"], p["n2"], p["b2"], EPS, stats=s["st2"])
    return s


def backward(canon, p, s, starts=None):
    n2 = canon.layer_norm_grad(p["dout"], s["sum"], p["n2"], s["st2"], p["b2"])
    r = canon.gated_recurrence_grad(n2.dx, s["u"], s["g"], s["keep"], p["decay"], s["i"], starts)
    c = canon.causal_conv_grad(r.dx, s["a"], p["conv"], p["cb"], "silu", starts)
    da = c.dx + r.dgate @ p["Wg"].t().contiguous() + r.dinput_gate @ p["Wi"].t().contiguous()
    n1 = canon.layer_norm_grad(da, s["x"], p["n1"], s["st1"], p["b1"], dsum=n2.dx)
    e = canon.embedding_grad(n1.dx, p["ids"], p["table"].shape[0], dtype=F32)
    return [e, n1.dweight, n1.dbias, c.dweight, c.dbias, r.ddecay, n2.dweight, n2.dbias]


NAMES = ["table", "n1", "b1", "conv", "cb", "decay", "n2", "b2"]


def plain(e, width=64):
    """The float64 form, with autograd."""
    def norm(x, w, b):
        return torch.nn.functional.layer_norm(x, (width,), w, b, EPS)

    x = e["table"][e["ids"]]
    a = norm(x, e["n1"], e["b1"])
    u = torch.stack([seq_ref.conv_one(r, e["conv"], e["cb"], True,
                                      torch.zeros(3, width).double())[0] for r in a])
    la = -e["decay"] * torch.sigmoid(a @ e["Wg"])
    v = torch.sqrt(-torch.expm1(2 * la)) * torch.sigmoid(a @ e["Wi"]) * u
    h = [torch.zeros_like(x[:, 0])]
    for t in range(x.shape[1]):
        h.append(torch.exp(la[:, t]) * h[-1] + v[:, t])
    return norm(torch.stack(h[1:], 1) + x, e["n2"], e["b2"])


def test_training_step(canon):
    """The output and every gradient against autograd of the float64 form, float32
    throughout.  Relative to each tensor's largest value: an output is 5 operators deep,
    with sums of 64 columns (norms, products) and 70 rows (the recurrence, of which each
    row rounds a few dozen times, as its own bounds count): 64 (70 + 64) roundings, twice
    that backward, times the 2^2 by which absolute sums of such inputs exceed the
    values."""
    p = model()
    s = forward(canon, p)
    got = backward(canon, p, s)
    e = {k: v.double().cpu() if v.is_floating_point() else v.cpu() for k, v in p.items()}
    for k in NAMES:
        e[k].requires_grad_()
    y = plain(e)
    want = torch.autograd.grad((y * e["dout"]).sum(), [e[k] for k in NAMES])
    bound = 4 * 2 * 64 * (70 + 64) * layer_ref.U
    for name, a, b in zip(["y"] + NAMES, [s["y"]] + got, [y.detach()] + list(want)):
        err = float((a.double().cpu() - b).abs().max() / b.abs().max())
        assert err <= bound, (name, err, bound)


def test_a_gradient_against_differences(canon):
    """The loss along a direction of the decays, the first norm's weights and the table,
    by central differences of the float64 form."""
    p = model(seqs=2, rows=40, seed=1)
    got = dict(zip(NAMES, backward(canon, p, forward(canon, p))))
    e = {k: v.double().cpu() if v.is_floating_point() else v.cpu() for k, v in p.items()}
    g = torch.Generator().manual_seed(5)
    for k in ("decay", "n1", "table"):
        d = torch.randn(e[k].shape, generator=g, dtype=torch.float64)
        step = 1e-5 * float(e[k].abs().max())
        loss = [float((plain(dict(e, **{k: e[k] + q * step * d})) * e["dout"]).sum())
                for q in (1, -1)]
        want = (loss[0] - loss[1]) / (2 * step)
        have = got[k].double().cpu() * d
        # the gradient's bound as above, for each component; the differences are off by
        # the square of the step
        bound = 4 * 2 * 64 * (40 + 64) * layer_ref.U * float(got[k].abs().max() * d.abs().sum())
        assert abs(float(have.sum()) - want) <= bound + 1e-6 * abs(want), k


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_generation(canon, dtype):
    """A prompt, then token after token: states continue, the norms' bits are the
    sequence's, the same numbers give the same tokens as the whole sequence read again."""
    p = model(dtype, vocab=211)
    prompt, width = p["ids"], 64
    conv = torch.empty(3, 3, width, dtype=dtype, device="cuda")
    state = torch.empty(3, width, device="cuda")
    s = forward(canon, p, conv, state)
    table = p["table"].t().contiguous()
    settings = dict(temperature=torch.tensor([0.0, 0.9, 1.3], device="cuda"),
                    top_k=torch.tensor([0, 40, 0], dtype=torch.int32, device="cuda"), top_p=0.95)
    u = torch.rand(12, 3, generator=torch.Generator().manual_seed(2)).cuda()
    nxt = canon.sample(s["y"][:, -1] @ table, u[0], **settings)
    told = []
    for t in range(1, 12):
        assert ((nxt >= 0) & (nxt < 211)).all()
        told.append(nxt)
        x = canon.embedding(p["table"], nxt)
        a = canon.layer_norm(x, p["n1"], p["b1"], EPS)
        c = canon.causal_conv_step(a, conv, p["conv"], p["cb"], "silu")
        h = canon.gated_recurrence_step(state, c, a @ p["Wg"], p["decay"], a @ p["Wi"])
        y, _ = canon.add_layer_norm(h, x, p["n2"], p["b2"], EPS)
        nxt = canon.sample(y @ table, u[t], **settings)
        # the same rows as part of the whole sequence
        q = dict(p, ids=torch.cat([prompt, torch.stack(told, 1)], 1))
        w = forward(canon, q)
        assert torch.equal(w["a"][:, -1], a) and torch.equal(w["u"][:, -1], c)
        # the products may differ in their last bits; both outputs are roundings of values
        # that close
        diff = (w["y"][:, -1].double() - y.double()).abs()
        half = torch.finfo(dtype).eps / 2
        assert (diff <= 64 * half * (1 + y.double().abs())).all()
    ref = (s["y"][:, -1] @ table).float().cpu().numpy()
    first = [layer_ref.sample(ref[i], float(u[0, i]), float(settings["temperature"][i]),
                              int(settings["top_k"][i]), 0.95) for i in range(3)]
    for i, (token, margin) in enumerate(first):
        assert margin < 1e-9 or int(told[0][i]) == token


def test_packed_sequences(canon):
    """Packed, the block's rows are those of the sequences alone, forward and back."""
    p = model(seqs=1, rows=70 + 1 + 33, seed=3)
    p["ids"], p["dout"] = p["ids"][0], p["dout"][0]
    starts = torch.tensor([0, 70, 70, 71, 104], dtype=torch.int32, device="cuda")
    s = forward(canon, p, starts=starts)
    n2 = canon.layer_norm_grad(p["dout"], s["sum"], p["n2"], s["st2"], p["b2"])
    r = canon.gated_recurrence_grad(n2.dx, s["u"], s["g"], s["keep"], p["decay"], s["i"], starts)
    for a, b in ((0, 70), (70, 71), (71, 104)):
        u, g, i, dout = (t[None, a:b] for t in (s["u"], s["g"], s["i"], n2.dx))
        keep = canon.gated_recurrence_states(u)
        h = canon.gated_recurrence(u, g, p["decay"], i, states=keep)
        alone = canon.gated_recurrence_grad(dout, u, g, keep, p["decay"], i)
        assert torch.equal(h[0], s["h"][a:b])
        for x, y in ((alone.dx, r.dx), (alone.dgate, r.dgate), (alone.dinput_gate, r.dinput_gate)):
            assert torch.equal(x[0], y[a:b])


def test_two_streams(canon):
    """Independent steps on two streams, each with its own buffers."""
    ps = [model(BF16, rows=600, width=256, seed=s) for s in (1, 2)]
    lg = [torch.randn(9, 5000, device="cuda") for _ in ps]
    us = [torch.rand(9, device="cuda") for _ in ps]

    def step(i):
        s = forward(canon, ps[i])
        return [s["y"]] + backward(canon, ps[i], s) + [canon.sample(lg[i], us[i], top_p=0.9)]

    want = [step(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    got = [None, None]
    for _ in range(3):
        for i in range(2):
            streams[i].wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(streams[i]):
                got[i] = step(i)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


# The operators alone in a graph: products are the library's.
def core(canon, q):
    st = canon.layer_norm_stats(q["x"])
    y, total = canon.add_layer_norm(q["x"], q["res"], q["w"], q["b"], EPS, stats=st)
    final, keep = torch.empty_like(q["init"]), canon.gated_recurrence_states(y)
    h = canon.gated_recurrence(y, q["gate"], q["decay"], q["inp"], None, q["init"], final, keep)
    r = canon.gated_recurrence_grad(q["dout"], y, q["gate"], keep, q["decay"], q["inp"])
    n = canon.layer_norm_grad(r.dx, total, q["w"], st, q["b"])
    ids = canon.sample(h.reshape(-1, h.shape[-1])[:40].contiguous(), q["u"], 0.8, q["k"], 0.9)
    return [y, h, final, ids, r.dx, r.dgate, r.dinput_gate, r.ddecay, r.dinit_state, n.dx,
            n.dweight, n.dbias]


def core_inputs(seed, seqs, rows, width):
    g = torch.Generator().manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, generator=g)

    p = {k: normal(seqs, rows, width).to(BF16) for k in ("x", "res", "gate", "inp", "dout")}
    p.update(w=normal(width), b=normal(width), decay=torch.rand(width, generator=g),
             init=normal(seqs, width), u=torch.rand(40, generator=g),
             k=torch.randint(0, 50, (40,), generator=g, dtype=torch.int32))
    return {k: v.cuda() for k, v in p.items()}


@pytest.mark.parametrize("seqs,rows,width", [(3, 130, 128), (2, 1100, 512), (30, 1100, 96),
                                            (50, 600, 320)])
def test_graph_capture(canon, seqs, rows, width):
    """One block, rounds side by side, blocks, whole sequences: captured, replayed on changed
    inputs with eager work and synchronisations between the replays."""
    p = core_inputs(3, seqs, rows, width)
    core(canon, p)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = core(canon, p)
    for seed in range(4):
        q = core_inputs(10 + seed, seqs, rows, width)
        for k in p:
            p[k].copy_(q[k])
        graph.replay()
        torch.cuda.synchronize()
        want = core(canon, q)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), seed


def test_decoding_in_a_graph(canon):
    """A decoding step captured with its states, replayed: every replay goes one row on."""
    q = core_inputs(7, 1, 6, 256)
    state, x = torch.zeros(5, 256, device="cuda"), torch.zeros(5, 256, dtype=BF16, device="cuda")
    rows = torch.randn(6, 5, 256, generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    u = torch.rand(5, device="cuda")

    def step(x, state):
        a = canon.layer_norm(x, q["w"], q["b"], EPS)
        h = canon.gated_recurrence_step(state, a, x, q["decay"], a)
        y, total = canon.add_layer_norm(h, x, q["w"], q["b"], EPS)
        return total, canon.sample(y, u, 1.1, 20)

    step(x, state)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x, state)
    state.zero_()
    eager = torch.zeros_like(state)
    for t in range(6):
        x.copy_(rows[t])
        graph.replay()
        torch.cuda.synchronize()
        want = step(rows[t], eager)
        assert all(torch.equal(a, b) for a, b in zip(out, want)), t
        assert torch.equal(state, eager)


def test_same_bits_every_run(canon):
    q = core_inputs(4, 4, 1300, 640)
    want = core(canon, q)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(core(canon, q), want))


@pytest.mark.parametrize("seqs", [2, 30, 100])
def test_workspaces_of_the_caller(canon, seqs):
    """A workspace of the caller's, larger than needed and full of other values, serves
    every call; one that is too small is left alone."""
    q = core_inputs(5, seqs, 1100, 96)
    want = core(canon, q)
    y, h = want[0], want[1]
    n = max(canon.gated_recurrence_workspace_bytes(seqs, 1100, False, 96),
            canon.gated_recurrence_grad_workspace_bytes(seqs, 1100, False, 96),
            canon.layer_norm_grad_workspace_bytes(seqs, 1100, 96))
    ws = torch.full((n + 64,), 0xff, dtype=torch.uint8, device="cuda")
    keep, st = canon.gated_recurrence_states(y), canon.layer_norm_stats(y)
    assert torch.equal(canon.gated_recurrence(y, q["gate"], q["decay"], q["inp"], None, q["init"],
                                              None, keep, ws=ws), h)
    r = canon.gated_recurrence_grad(q["dout"], y, q["gate"], keep, q["decay"], q["inp"], ws=ws)
    assert torch.equal(r.dx, want[4]) and torch.equal(r.ddecay, want[7])
    _, total = canon.add_layer_norm(q["x"], q["res"], q["w"], q["b"], EPS, stats=st)
    g = canon.layer_norm_grad(r.dx, total, q["w"], st, q["b"], ws=ws)
    assert torch.equal(g.dx, want[9]) and torch.equal(g.dweight, want[10])
    small = torch.full_like(ws[:16], 0xff)  # the call allocates its own
    r = canon.gated_recurrence_grad(q["dout"], y, q["gate"], keep, q["decay"], q["inp"], ws=small)
    assert torch.equal(r.dx, want[4]) and (small == 0xff).all()
    with pytest.raises(ValueError):
        canon.layer_norm_grad(r.dx, total, q["w"], st, q["b"], ws=ws.view(torch.int8))
