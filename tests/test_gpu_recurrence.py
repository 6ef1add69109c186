"""The gated linear recurrence against its float64 form: forward, backward, single
rows, packing and cutting."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import layer_ref  # noqa: E402

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
BLOCK = layer_ref.BLOCK


@pytest.fixture(scope="module")
def canon():
    import scan_canonical_reduce_amd as c
    return c


def inputs(dtype, lens, channels, packed=False, decay=True, gated=True, seed=0, before=0,
           after=0, slow=False):
    """before, after: packed rows that belong to no sequence; slow: a close to 1."""
    g = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g)

    lead = (before + sum(lens) + after,) if packed else (len(lens), lens[0])
    d = dict(x=normal(*lead, channels).to(dtype), gate=(1.5 * normal(*lead, channels)).to(dtype),
             input_gate=normal(*lead, channels).to(dtype) if gated else None,
             decay=torch.rand(channels, generator=g) * (0.01 if slow else 0.5) if decay else None,
             init=normal(len(lens), channels), dfinal=normal(len(lens), channels),
             dout=normal(*lead, channels).to(dtype),
             starts=(torch.tensor([0] + lens).cumsum(0) + before).int() if packed else None)
    return {k: v.cuda() if torch.is_tensor(v) else v for k, v in d.items()}


GATES = ("x", "gate", "input_gate")


def forward(canon, d, init=True, **kw):
    return canon.gated_recurrence(d["x"], d["gate"], d["decay"], d["input_gate"], d["starts"],
                                  d["init"] if init else None, **kw)


def backward(canon, d, states, dfinal=True):
    return canon.gated_recurrence_grad(d["dout"], d["x"], d["gate"], states, d["decay"],
                                       d["input_gate"], d["starts"],
                                       d["dfinal"] if dfinal else None)


def pieces(d):
    """(rows of the leading dimension or sequences, inputs of the float64 form) for sets
    of sequences of one length"""
    if d["starts"] is None:
        return [(slice(None), slice(None), {k: d[k] for k in GATES + ("dout",)})]
    p = d["starts"].tolist()
    return [(slice(a, b), slice(i, i + 1),
             {k: None if d[k] is None else d[k][a:b][None] for k in GATES + ("dout",)})
            for i, (a, b) in enumerate(zip(p, p[1:]))]


def check(canon, d, grad=True, init=True, dfinal=True):
    final = torch.full_like(d["init"], 7.0)
    states = canon.gated_recurrence_states(d["x"], d["starts"])
    out = torch.full_like(d["x"], 7.0)
    got = forward(canon, d, init, final_state=final, states=states, out=out)
    assert got is out
    g = backward(canon, d, states, dfinal) if grad else None
    ddecay, bound = 0, 0
    for rows, seqs, part in pieces(d):
        dout = part.pop("dout")
        r = layer_ref.recur(**part, decay=d["decay"], init=d["init"][seqs] if init else None,
                            dout=dout if grad else None,
                            dfinal=d["dfinal"][seqs] if dfinal else None)

        def of(t):
            return t[rows] if d["starts"] is None else t[rows][None]

        layer_ref.within(of(got), *r["out"], "out")
        layer_ref.within(final[seqs], *r["final"], "final")
        if not grad:
            continue
        layer_ref.within(of(g.dx), *r["x"], "dx")
        layer_ref.within(of(g.dgate), *r["gate"], "dgate")
        if d["input_gate"] is not None:
            layer_ref.within(of(g.dinput_gate), *r["input_gate"], "dinput_gate")
        layer_ref.within(g.dinit_state[seqs], *r["init"], "dinit_state")
        if d["decay"] is not None:
            ddecay, bound = ddecay + r["decay"][0], bound + r["decay"][1]
    if grad and d["decay"] is not None:
        # the sum over the sequences: at most one more rounding each of the bound's sums
        layer_ref.within(g.ddecay, ddecay, bound * 2, "ddecay")
    if d["starts"] is not None:
        p = d["starts"].tolist()
        assert (got[:p[0]] == 7).all() and (got[p[-1]:] == 7).all()
    return got, final, g


KINDS = [(True, True), (True, False), (False, True), (False, False)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("decay,gated", KINDS)
@pytest.mark.parametrize("channels", [1, 63, 64, 65, 200])
def test_short(canon, dtype, decay, gated, channels):
    for lens in ([1], [15, 15], [16], [17, 17, 17], [129], [300, 300]):
        check(canon, inputs(dtype, lens, channels, False, decay, gated, channels + lens[0]))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("decay,gated", KINDS)
def test_packed(canon, dtype, decay, gated):
    for lens in ([5, 0, 64, 1, 31, 0, 2, 100], [0], [0, 0], [512], [1]):
        check(canon, inputs(dtype, lens, 70, True, decay, gated, sum(lens), before=3, after=6))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("decay,gated", [(True, True), (False, False)])
def test_blocks(canon, dtype, decay, gated):
    """More than one block of a sequence: in three launches."""
    for lens in ([511], [512], [513], [1024, 1024], [1500]):
        check(canon, inputs(dtype, lens, 66, False, decay, gated, lens[0], slow=True))
    check(canon, inputs(dtype, [700, 0, 513, 512, 1, 1300, 0], 66, True, decay, gated, 9, 2, 5,
                        slow=True))
    check(canon, inputs(dtype, [2600], 8, False, decay, gated, 11), init=False, dfinal=False)


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("decay,gated", [(True, True), (False, False)])
def test_whole_sequences(canon, dtype, decay, gated):
    """A workgroup per sequence and slab."""
    check(canon, inputs(dtype, [1100] * 260, 20, False, decay, gated, 5))
    check(canon, inputs(dtype, [530] * 16, 1100, False, decay, gated, 6), init=False, dfinal=False)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_large_decays(canon, dtype):
    """Decays from 0 to 100, 1 and its neighbours among them: in waves of channels with
    none above 1, with some, and with large ones only."""
    small = [0.0, 1e-6, 0.01, 0.35, 0.9, 1 - 2.0 ** -24, 1.0]
    large = [1 + 2.0 ** -23, 1.5, 3.0, 8.0, 30.0, 100.0]
    decay = torch.tensor((small * 19)[:128] + (small + large) * 10 + large * 20)
    for lens in ([200] * 2, [600]):
        d = inputs(dtype, lens, len(decay), seed=lens[0])
        d["decay"] = decay.cuda()
        check(canon, d)
    d = inputs(dtype, [1] * 5, len(decay), seed=2)
    d["decay"] = decay.cuda()
    r = layer_ref.recur(d["x"], d["gate"], d["input_gate"], d["decay"], d["init"])
    state = d["init"].clone()
    out = canon.gated_recurrence_step(state, d["x"][:, 0], d["gate"][:, 0], d["decay"],
                                      d["input_gate"][:, 0])
    layer_ref.within(out[:, None], *r["out"], "out")
    layer_ref.within(state, *r["final"], "state")


def test_a_long_memory(canon):
    """a of 0.9999 and more over 9000 rows in float32."""
    for lens, packed in (([9000], False), ([3000, 6000], True)):
        d = inputs(F32, lens, 6, packed, slow=True, seed=4)
        d["decay"] *= 0.02
        check(canon, d)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("decay", [False, True])
def test_same_bits_however_it_is_spread(canon, dtype, decay):
    """Alone or with others, packed or not, whole or in blocks, cut at whole blocks."""
    n, rows, ch = 300, 2 * BLOCK + 77, 24
    d = inputs(dtype, [rows] * n, ch, decay=decay)  # whole: 300 workgroups
    final = torch.empty_like(d["init"])
    states = canon.gated_recurrence_states(d["x"])
    out = forward(canon, d, final_state=final, states=states)
    g = backward(canon, d, states)
    pick = slice(41, 44)

    def part(rows_=slice(None), seqs=pick):
        return {k: v if v is None or k in ("decay", "starts") else
                v[seqs].contiguous() if k in ("init", "dfinal") else v[seqs, rows_]
                for k, v in d.items()}

    p = part()  # in blocks: 3 sequences of one slab
    f2, s2 = torch.empty_like(p["init"]), canon.gated_recurrence_states(p["x"])
    o2 = forward(canon, p, final_state=f2, states=s2)
    assert torch.equal(o2, out[pick]) and torch.equal(f2, final[pick])
    g2 = backward(canon, p, s2)
    for a, b in zip((g2.dx, g2.dgate, g2.dinput_gate, g2.dinit_state),
                    (g.dx, g.dgate, g.dinput_gate, g.dinit_state)):
        assert torch.equal(a, b[pick])
    # packed, with an empty sequence among them
    q = dict(p, starts=torch.tensor([1, 1 + rows, 1 + 2 * rows, 1 + 2 * rows, 1 + 3 * rows],
                                    dtype=torch.int32, device="cuda"))
    for k in GATES + ("dout",):
        q[k] = torch.cat([torch.zeros_like(p[k][0, :1]), p[k].reshape(-1, ch)])
    for k in ("init", "dfinal"):
        q[k] = torch.cat([p[k][:2], torch.ones_like(p[k][:1]), p[k][2:]])
    f3, s3 = torch.empty_like(q["init"]), canon.gated_recurrence_states(q["x"], q["starts"])
    o3 = forward(canon, q, final_state=f3, states=s3)
    assert torch.equal(o3[1:], o2.reshape(-1, ch)) and torch.equal(f3[[0, 1, 3]], f2)
    assert (f3[2] == 1).all()
    g3 = backward(canon, q, s3)
    for a, b in zip(g3[:2] + (g3.dinput_gate,), g2[:2] + (g2.dinput_gate,)):
        assert torch.equal(a[1:], b.reshape(-1, ch))
    assert torch.equal(g3.dinit_state[[0, 1, 3]], g2.dinit_state)
    # cut
    for cut in (BLOCK, 2 * BLOCK):
        a, b = part(slice(0, cut)), part(slice(cut, rows))
        state = a["init"].clone()
        oa = forward(canon, a, final_state=state)
        b["init"] = state
        ob = forward(canon, b, final_state=state)
        assert torch.equal(torch.cat([oa, ob], 1), o2) and torch.equal(state, f2)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_same_bits_with_any_number_of_sequences(canon, dtype):
    """Whole with two channels a lane where they fit, and with one; in blocks so and
    so; 2 blocks and a row, an even and an odd number of channels."""
    for ch in (130, 129):
        d = inputs(dtype, [2 * BLOCK + 1] * 110, ch, seed=ch)
        d["decay"][5], d["decay"][100] = 1.0, 3.0  # one alone in some waves, not in others
        d["gate"][:, ::10, 5] = 40.0
        for k in GATES + ("init", "dfinal", "dout"):
            d[k] = torch.cat([d[k]] * 2)
        want = None
        for n in (220, 80, 64, 3, 1):  # 3 slabs of 64 channels each
            p = {k: v if v is None or k in ("decay", "starts") else v[:n] for k, v in d.items()}
            final, states = torch.empty_like(p["init"]), canon.gated_recurrence_states(p["x"])
            got = [forward(canon, p, final_state=final, states=states), final]
            g = backward(canon, p, states)
            got += [g.dx, g.dgate, g.dinput_gate, g.dinit_state]
            if want is None:
                want = got
            assert all(torch.equal(a, b[:n]) for a, b in zip(got, want)), (ch, n)
        assert all(torch.equal(t[:110], t[110:]) for t in want)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows", [257, 384, 500, 512, 1000, 7 * BLOCK + 130])
def test_same_bits_by_rounds(canon, dtype, rows):
    """Few sequences, whose rounds have a workgroup each, and many, packed or not; the
    decays' gradients within the sums' roundings."""
    few, ch = 2, 68
    d = inputs(dtype, [rows] * (40 if rows > BLOCK else 70), ch, seed=rows)
    out, g, final = [], [], []
    for n in (len(d["x"]), few):
        p = {k: v if v is None or k in ("decay", "starts") else v[:n] for k, v in d.items()}
        final.append(torch.empty_like(p["init"]))
        states = canon.gated_recurrence_states(p["x"])
        out.append(forward(canon, p, final_state=final[-1], states=states))
        g.append(backward(canon, p, states))
    p["starts"] = torch.tensor([0, rows, rows, 2 * rows], dtype=torch.int32, device="cuda")
    for k in GATES + ("dout",):
        p[k] = p[k].reshape(-1, ch)
    for k in ("init", "dfinal"):
        p[k] = torch.cat([p[k][:1], torch.full_like(p[k][:1], 3.0), p[k][1:]])
    state, states = p["init"].clone(), canon.gated_recurrence_states(p["x"], p["starts"])
    h = canon.gated_recurrence(p["x"], p["gate"], p["decay"], p["input_gate"], p["starts"], state,
                               state, states)
    b = backward(canon, p, states)
    assert torch.equal(out[1], out[0][:few]) and torch.equal(final[1], final[0][:few])
    assert torch.equal(h.reshape(out[1].shape), out[1]) and torch.equal(state[[0, 2]], final[1])
    assert (state[1] == 3).all() and (b.dinit_state[1] == 3).all()
    assert torch.equal(b.dinit_state[[0, 2]], g[1].dinit_state)
    for name in ("dx", "dgate", "dinput_gate", "dinit_state"):
        one = getattr(g[1], name)
        assert torch.equal(one, getattr(g[0], name)[:few])
        if name != "dinit_state":
            assert torch.equal(getattr(b, name).reshape(one.shape), one)
    # the sum over a few thousand rows in two orders: gate's gradient is its term times
    # decay (1 - sigmoid(gate)), so the absolute sum is at most that of |dgate| over it
    share = (d["decay"] * torch.sigmoid(-d["gate"][:few].double())).clamp(min=1e-9)
    size = (g[1].dgate.double().abs() / share).sum((0, 1)) + 1e-3
    bound = 2 * (128 + 64) * layer_ref.U * size * (1 + 2 ** -7)
    assert ((g[1].ddecay.double() - b.ddecay.double()).abs() <= bound).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("packed", [False, True])
def test_many_blocks(canon, dtype, packed):
    """More blocks than each folds those before it: the same bits, forward and backward,
    as two calls that pass the state and its gradient on."""
    blocks, cut = 35, 17 * BLOCK
    d = inputs(dtype, [blocks * BLOCK - 100], 6, packed, slow=True, seed=8)
    final, states = torch.empty_like(d["init"]), canon.gated_recurrence_states(d["x"], d["starts"])
    out = forward(canon, d, final_state=final, states=states)
    g = backward(canon, d, states)
    rows = (lambda t, s: t[s]) if packed else (lambda t, s: t[:, s])
    parts, state = [], d["init"]
    for s in (slice(0, cut), slice(cut, None)):
        p = dict(d, init=state, **{k: rows(d[k], s).contiguous() for k in GATES + ("dout",)})
        if packed:
            p["starts"] = torch.tensor([0, p["x"].shape[0]], dtype=torch.int32, device="cuda")
        state, keep = torch.empty_like(state), canon.gated_recurrence_states(p["x"], p["starts"])
        assert torch.equal(forward(canon, p, final_state=state, states=keep), rows(out, s))
        parts.append((s, p, keep))
    assert torch.equal(state, final)
    dfinal = d["dfinal"]
    for s, p, keep in reversed(parts):
        b = backward(canon, dict(p, dfinal=dfinal), keep)
        dfinal = b.dinit_state
        for x, y in ((b.dx, g.dx), (b.dgate, g.dgate), (b.dinput_gate, g.dinput_gate)):
            assert torch.equal(x, rows(y, s))
    assert torch.equal(dfinal, g.dinit_state)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("decay,gated", KINDS)
def test_step(canon, dtype, decay, gated):
    for n, channels in ((1, 1), (3, 65), (37, 264), (5, 1024)):
        d = inputs(dtype, [1] * n, channels, False, decay, gated, n)
        row = {k: None if d[k] is None else d[k][:, 0] for k in GATES}
        r = layer_ref.recur(**{k: d[k] for k in GATES}, decay=d["decay"], init=d["init"])
        nxt = torch.empty_like(d["init"])
        got = canon.gated_recurrence_step(d["init"], row["x"], row["gate"], d["decay"],
                                          row["input_gate"], out_state=nxt)
        layer_ref.within(got, r["out"][0][:, 0], r["out"][1][:, 0], "out")
        layer_ref.within(nxt, *r["final"], "state")
        state = d["init"].clone()
        again = canon.gated_recurrence_step(state, row["x"], row["gate"], d["decay"],
                                            row["input_gate"], out=torch.empty_like(got))
        assert torch.equal(again, got) and torch.equal(state, nxt)


def test_step_strided(canon):
    """Rows of a larger buffer, odd pitch and start."""
    d = inputs(BF16, [1] * 9, 130, seed=2)
    want = canon.gated_recurrence_step(d["init"].clone(), d["x"][:, 0], d["gate"][:, 0], d["decay"],
                                       d["input_gate"][:, 0])
    big = torch.full((9, 3 * 131 + 1), 7.0, dtype=BF16, device="cuda")
    views = [big[:, 1 + i * 131:131 + i * 131] for i in range(3)]
    for v, k in zip(views, GATES):
        v.copy_(d[k][:, 0])
    out = torch.full((9, 133), 7.0, dtype=BF16, device="cuda")
    canon.gated_recurrence_step(d["init"].clone(), views[0], views[1], d["decay"], views[2],
                                out=out[:, 2:132])
    assert torch.equal(out[:, 2:132], want)
    assert (out[:, :2] == 7).all() and (out[:, 132:] == 7).all()


def test_decoding_continues_the_prompt(canon):
    """A prompt, then single rows: both within the bound of the whole sequence."""
    d = inputs(BF16, [90] * 3, 70, seed=8)
    cut, state = 61, d["init"].clone()
    p = {k: v if v is None or k in ("decay", "init", "dfinal", "starts") else v[:, :cut]
         for k, v in d.items()}
    outs = [forward(canon, p, final_state=state)]
    for t in range(cut, 90):
        outs.append(canon.gated_recurrence_step(state, d["x"][:, t], d["gate"][:, t], d["decay"],
                                                d["input_gate"][:, t])[:, None])
    r = layer_ref.recur(**{k: d[k] for k in GATES}, decay=d["decay"], init=d["init"])
    layer_ref.within(torch.cat(outs, 1), *r["out"], "out")
    layer_ref.within(state, *r["final"], "state")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strides(canon, dtype):
    """Views of wider, unaligned buffers, sequences interleaved, broadcast inputs."""
    d = inputs(dtype, [150] * 4, 67, seed=3)
    states = canon.gated_recurrence_states(d["x"])
    want = forward(canon, d, states=states)
    grads = backward(canon, d, states)
    e = dict(d)
    for k in GATES + ("dout",):
        big = torch.zeros(150, 4, 75, dtype=dtype, device="cuda")
        v = big.transpose(0, 1)[:, :, 5:72]
        v.copy_(d[k])
        e[k] = v
    out = torch.full((150, 4, 75), 7.0, dtype=dtype, device="cuda")
    forward(canon, e, out=out.transpose(0, 1)[:, :, 1:68])
    assert torch.equal(out.transpose(0, 1)[:, :, 1:68], want)
    assert (out[..., :1] == 7).all() and (out[..., 68:] == 7).all()
    assert all(torch.equal(a, b) for a, b in zip(backward(canon, e, states), grads))
    e = dict(d, gate=d["gate"][:1, :1].expand(4, 150, 67), x=d["x"][:1].expand(4, 150, 67))
    f = {k: v.contiguous() if k in GATES else v for k, v in e.items()}
    assert torch.equal(forward(canon, e), forward(canon, f))


def test_final_state_in_place(canon):
    """final_state may be init_state, also where the blocks run side by side."""
    for lens, ch, packed in (([90] * 3, 64, False), ([5000], 40, False), ([1100] * 260, 20, False),
                             ([700, 0, 2000], 64, True)):
        d = inputs(F32, lens, ch, packed)
        want = torch.empty_like(d["init"])
        out = forward(canon, d, final_state=want)
        state = d["init"].clone()
        got = canon.gated_recurrence(d["x"], d["gate"], d["decay"], d["input_gate"], d["starts"],
                                     state, state)
        assert torch.equal(got, out) and torch.equal(state, want)


def test_gates_at_their_limits(canon):
    """Gates of plus and minus infinity, and a decay of zero, are limits: the state is
    kept or replaced, and gradients are finite."""
    inf = float("inf")
    for decay in (False, True):
        d = inputs(F32, [40] * 2, 64, decay=decay, gated=False)
        keep = -inf if decay else inf  # an a of 1
        d["gate"][:, 10:20] = keep
        d["gate"][:, 30] = -keep
        if decay:
            d["decay"][:8] = 0.0
        states = canon.gated_recurrence_states(d["x"])
        out = forward(canon, d, states=states)
        assert torch.isfinite(out).all()
        # kept inside a chunk of 8 rows; the next one starts from its own carry
        assert (out[:, 10:16] == out[:, 9:10]).all() and (out[:, 17:20] == out[:, 16:17]).all()
        if decay:
            assert (out[..., :8] == d["init"][:, None, :8]).all()
        g = backward(canon, d, states)
        assert all(torch.isfinite(t).all() for t in g if t is not None)
        r = layer_ref.recur(d["x"], d["gate"].clamp(-80, 80), None, d["decay"], d["init"],
                            d["dout"], d["dfinal"])
        layer_ref.within(out, *r["out"], "out")


def test_what_is_not_finite_stays_in_its_channel(canon):
    for lens, ch in (([700] * 2, 66), ([1100] * 260, 20)):
        d = inputs(F32, lens, ch)
        want = forward(canon, d)
        for bad in (float("nan"), float("inf")):
            e = dict(d, x=d["x"].clone())
            e["x"][1, 530, 3] = bad
            got = forward(canon, e)
            assert not torch.isfinite(got[1, 530:, 3]).any()
            got[1, 530:, 3] = want[1, 530:, 3]
            assert torch.equal(got, want)


@pytest.mark.parametrize("rows", [0, 5, 600, 1500])
def test_rows_of_no_sequence(canon, rows):
    starts = torch.tensor([2], dtype=torch.int32, device="cuda")
    x = torch.randn(rows, 40, device="cuda")
    decay = torch.rand(40, device="cuda")
    out = torch.full_like(x, 7.0)
    keep = canon.gated_recurrence_states(x, starts)
    canon.gated_recurrence(x, x.clone(), decay, None, starts, states=keep, out=out)
    assert (out == 7).all()
    g = canon.gated_recurrence_grad(x, x, x, keep, decay, x, starts)
    assert not g.ddecay.any() and g.dinit_state.shape == (0, 40)


def test_starts_beyond_the_rows(canon):
    """Values outside [0, rows] count as the nearest, descending ones as empty."""
    d = inputs(F32, [600, 600], 33, True)
    d["starts"] = torch.tensor([-5, 600, 4000], dtype=torch.int32, device="cuda")
    want = forward(canon, inputs(F32, [600, 600], 33, True))
    assert torch.equal(forward(canon, d), want)
    d["starts"] = torch.tensor([600, 0, 1200], dtype=torch.int32, device="cuda")
    out = forward(canon, d)
    assert torch.isfinite(out).all()


def test_refusals(canon):
    d = inputs(F32, [4] * 2, 16)
    x, gate, decay = d["x"], d["gate"], d["decay"]
    states = canon.gated_recurrence_states(x)
    for call, kind in (
            (lambda: canon.gated_recurrence(x[0], gate[0]), ValueError),
            (lambda: canon.gated_recurrence(x.double(), gate.double()), TypeError),
            (lambda: canon.gated_recurrence(x, gate.half()), ValueError),
            (lambda: canon.gated_recurrence(x, gate[:1]), ValueError),
            (lambda: canon.gated_recurrence(x, gate, decay.half()), ValueError),
            (lambda: canon.gated_recurrence(x, gate, decay[:8]), ValueError),
            (lambda: canon.gated_recurrence(x, gate, init_state=d["init"][:1]), ValueError),
            (lambda: canon.gated_recurrence(x, gate, states=states[:-1]), ValueError),
            (lambda: canon.gated_recurrence(x, gate, out=x), ValueError),
            (lambda: canon.gated_recurrence(x, gate, starts=torch.tensor([0, 2])), ValueError),
            (lambda: canon.gated_recurrence(x, gate, decay.cpu()), ValueError),
            (lambda: canon.gated_recurrence_grad(x, x, gate, states[:-1]), ValueError),
            (lambda: canon.gated_recurrence_step(d["init"], x, gate), ValueError),
            (lambda: canon.gated_recurrence_step(d["init"][:1], x[:, 0], gate[:, 0]), ValueError)):
        with pytest.raises(kind):
            call()
