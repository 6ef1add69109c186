"""Selective scan against its float64 form: forward, backward, single rows."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import seq_ref  # noqa: E402
from gpu_util import launches  # noqa: E402

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def canon():
    import scan_canonical_reduce_amd as c
    return c


def inputs(dtype, lens, channels, groups, states, packed, seed=0):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g)

    lead = (sum(lens),) if packed else (len(lens), lens[0])
    return dict(
        u=normal(*lead, channels).to(dtype), delta=(normal(*lead, channels) * 0.7).to(dtype),
        z=normal(*lead, channels).to(dtype), B=normal(*lead, groups, states).to(dtype),
        C=normal(*lead, groups, states).to(dtype),
        A=-torch.exp(normal(channels, states)), D=normal(channels),
        bias=torch.rand(channels, generator=g) * 4 - 5,
        init=normal(len(lens), channels, states), dout=normal(*lead, channels).to(dtype),
        dfinal=normal(len(lens), channels, states),
        starts=torch.tensor([0] + lens).cumsum(0).int() if packed else None)


def cuda(d):
    return {k: v.cuda() if torch.is_tensor(v) else v for k, v in d.items()}


def call(canon, d, full=True, **kw):
    """selective_scan of everything (full), or of the plainest arguments."""
    if full:
        kw = dict(D=d["D"], z=d["z"], delta_bias=d["bias"], delta_softplus=True,
                  init_state=d["init"], **kw)
    return canon.selective_scan(d["u"], d["delta"] if full else d["delta"].abs(), d["A"], d["B"],
                                d["C"], starts=d["starts"], **kw)


def reference(d, full=True, leaves=None, absolute=False):
    """float64 out and final state; with `absolute`, of the absolute terms."""
    e = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v
         for k, v in d.items()}
    if leaves is not None:
        for k in leaves:
            e[k].requires_grad_()
    u, B, C, D, init = (e[k].abs() if absolute else e[k] for k in ("u", "B", "C", "D", "init"))
    outs, finals = [], []
    for i, at in enumerate(seq_ref.spans(d["u"], d["starts"])):
        z = e["z"][at] if full else None
        y, h = seq_ref.scan_one(u[at], e["delta"][at] if full else e["delta"][at].abs(), e["A"],
                                B[at], C[at], D if full else None, None if absolute else z,
                                e["bias"] if full else None, full,
                                init[i] if full else torch.zeros_like(init[i]))
        if absolute and full:
            y = y * z.abs()
        outs.append(y), finals.append(h)
    out = (torch.stack if d["starts"] is None else torch.cat)(outs)
    return out, torch.stack(finals), e


# One step multiplies by a = exp2(dl A log2 e): two rounded products and the
# hardware's exponential, at most 2 |log a| + 2 roundings of relative error, and
# adds dl u B, three products and a softplus within 10 roundings; it rounds
# twice.  A term that is still there after r more steps has been multiplied by
# prod a = exp(-X), X = sum |log a|, so that its errors of 2 X roundings, and of
# 10 X from dl's own, weigh at most 12 X exp(-X) <= 5; the other 4 per step add
# up to 4 rows.  Sums over at most 16 states, D u and the gate add less than 40,
# the start states of chunks 4 for each 64 rows.
def terms(rows):
    return 5 * rows + 64


SHAPES = [  # lens, channels, groups, states, packed
    ([1], 1, 1, 1, False), ([1, 1], 16, 1, 16, False), ([17, 17], 40, 2, 16, False),
    ([64], 64, 1, 16, False), ([65], 65, 1, 8, False), ([130], 96, 3, 13, False),
    ([200, 200], 72, 1, 5, False), ([150], 20, 1, 3, False), ([129], 130, 1, 4, False),
    ([3, 0, 64, 1, 129, 63, 0], 40, 1, 16, True), ([100, 65, 0, 1], 36, 2, 7, True),
    ([0, 0, 5], 17, 1, 2, True), ([30, 0, 64, 1, 33], 40, 1, 16, True), ([0, 65, 0, 62, 0], 70, 2, 8, True),
    ([128, 128], 24, 1, 16, False),
]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("lens,channels,groups,states,packed", SHAPES)
def test_forward(canon, dtype, lens, channels, groups, states, packed):
    d = inputs(dtype, lens, channels, groups, states, packed, channels + states)
    g = cuda(d)
    n = terms(max(lens))
    for full in (True, False):
        final = torch.full_like(g["init"], 7.0)
        got = call(canon, g, full, final_state=final)
        out, h, _ = reference(d, full)
        size, hsize, _ = reference(d, full, absolute=True)
        seq_ref.close(got, out, size, n, (lens, full, "out"))
        seq_ref.close(final, h, hsize, n, (lens, full, "final"))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("lens,channels,groups,states,packed", SHAPES)
def test_backward(canon, dtype, lens, channels, groups, states, packed):
    """Against autograd of the float64 form.  The bound's sums of absolute
    terms: autograd of the same form with every term positive (absolute inputs
    and incoming gradients), whose error terms are those of the forward pass
    twice (h and lam are such sums), and one per row and channel added."""
    d = inputs(dtype, lens, channels, groups, states, packed, 3 * channels + states)
    g = cuda(d)
    for full in (True, False):
        keep = canon.selective_scan_states(g["u"], states, g["starts"])
        call(canon, g, full, states=keep)
        kw = dict(D=g["D"], z=g["z"], delta_bias=g["bias"], delta_softplus=True,
                  d_final_state=g["dfinal"]) if full else {}
        delta = g["delta"] if full else g["delta"].abs()
        got = canon.selective_scan_grad(g["dout"], g["u"], delta, g["A"], g["B"], g["C"], keep,
                                        starts=g["starts"], **kw)
        names = ["u", "delta", "A", "B", "C"] + (["D", "z", "bias", "init"] if full else [])
        mine = [got.du, got.ddelta, got.dA, got.dB, got.dC] + (
            [got.dD, got.dz, got.ddelta_bias, got.dinit_state] if full else [])
        ref = {**d, "delta": d["delta"] if full else d["delta"].abs()}
        out, h, e = reference(ref, full, leaves=names)
        loss = (out * e["dout"]).sum() + ((h * e["dfinal"]).sum() if full else 0)
        want = torch.autograd.grad(loss, [e[k] for k in names], allow_unused=True)
        size = grad_sizes(ref, full, names)
        rows = max(lens)
        for k, a, b in zip(names, mine, want):
            b = torch.zeros_like(e[k]) if b is None else b
            extra = sum(lens) if k in ("A", "D", "bias") else channels
            seq_ref.close(a, b, size[k], 2 * terms(rows) + extra, (lens, full, k))


def grad_sizes(d, full, names):
    """Sums of absolute terms of each gradient, by the formulas."""
    e = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v
         for k, v in d.items()}
    res = {k: torch.zeros_like(e[k]) for k in names}
    for i, at in enumerate(seq_ref.spans(d["u"], d["starts"])):
        u, B, C = e["u"][at].abs(), e["B"][at].abs(), e["C"][at].abs()
        raw = e["delta"][at] + (e["bias"] if full else 0)
        dl = torch.nn.functional.softplus(raw, threshold=1e9) if full else raw
        slope = torch.sigmoid(raw) if full else torch.ones_like(raw)
        per = u.shape[1] // B.shape[1]
        Bf, Cf = B.repeat_interleave(per, 1), C.repeat_interleave(per, 1)
        a = torch.exp(dl[..., None] * e["A"])
        h = [e["init"][i].abs() if full else torch.zeros_like(e["init"][i])]
        for t in range(u.shape[0]):
            h.append(a[t] * h[-1] + (dl[t] * u[t])[:, None] * Bf[t])
        go = e["dout"][at].abs()
        z = e["z"][at].abs() if full else torch.ones_like(u)
        dy = go * z
        R = e["dfinal"][i].abs() if full else torch.zeros_like(h[0])
        for t in range(u.shape[0] - 1, -1, -1):
            idx = at[0].start + t if isinstance(at[0], slice) else (at[0], t)
            lam = Cf[t] * dy[t][:, None] + R
            R = a[t] * lam
            dec = R * h[t]
            thr = (lam * Bf[t]).sum(-1)
            res["u"][idx] = thr * dl[t] + (e["D"].abs() * dy[t] if full else 0)
            dd = ((dec * e["A"].abs()).sum(-1) + thr * u[t]) * slope[t]
            res["delta"][idx] = dd
            res["A"] += dec * dl[t][:, None]
            G = B.shape[1]
            res["B"][idx] = (lam * (dl[t] * u[t])[:, None]).view(G, per, -1).sum(1)
            res["C"][idx] = (h[t + 1] * dy[t][:, None]).view(G, per, -1).sum(1)
            if full:
                y = (h[t + 1] * Cf[t]).sum(-1) + e["D"].abs() * u[t]
                res["D"] += dy[t] * u[t]
                res["bias"] += dd
                res["z"][idx] = go[t] * y * (1.1 + z[t])
        if full:
            res["init"][i] = R
    return res


def test_backward_against_differences(canon):
    """<gradient, v> against a central difference of the float64 form along v;
    float32 rows of 1e-6 relative error summed, and the step's 1e-10."""
    d = inputs(F32, [70, 0, 9], 20, 2, 6, True, 5)
    g = cuda(d)
    keep = canon.selective_scan_states(g["u"], 6, g["starts"])
    call(canon, g, states=keep)
    got = canon.selective_scan_grad(
        g["dout"], g["u"], g["delta"], g["A"], g["B"], g["C"], keep, D=g["D"], z=g["z"],
        delta_bias=g["bias"], delta_softplus=True, starts=g["starts"], d_final_state=g["dfinal"])
    for key, grad in (("u", got.du), ("delta", got.ddelta), ("A", got.dA), ("B", got.dB),
                      ("C", got.dC), ("D", got.dD), ("z", got.dz), ("bias", got.ddelta_bias),
                      ("init", got.dinit_state)):
        v = torch.randn(d[key].shape, generator=torch.Generator().manual_seed(1)).double()

        def f(step):
            e = {k: t.double() if torch.is_tensor(t) and t.is_floating_point() else t
                 for k, t in d.items()}
            e[key] = e[key] + step * v
            out, h, _ = reference(e)
            return float((out * e["dout"]).sum() + (h * e["dfinal"]).sum())

        want = (f(1e-5) - f(-1e-5)) / 2e-5
        assert float((grad.double().cpu() * v).sum()) == pytest.approx(want, rel=1e-4, abs=1e-3)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_bits_of_packing_batch_and_pieces(canon, dtype):
    """A sequence's bits do not depend on the batch, on packing, or on being
    cut at multiples of 64 rows with the state handed on."""
    d = cuda(inputs(dtype, [300] * 3, 80, 1, 16, False, 2))
    final = torch.empty_like(d["init"])
    want = call(canon, d, final_state=final)
    alone = {k: v[1:2].contiguous() if k not in ("A", "D", "bias", "starts") else v
             for k, v in d.items()}
    f1 = torch.empty_like(alone["init"])
    assert torch.equal(call(canon, alone, final_state=f1), want[1:2])
    assert torch.equal(f1, final[1:2])
    packed = {k: v.flatten(0, 1) if k in ("u", "delta", "z", "B", "C") else v
              for k, v in d.items()}
    packed["starts"] = torch.tensor([0, 300, 600, 900]).int().cuda()
    f2 = torch.empty_like(final)
    assert torch.equal(call(canon, packed, final_state=f2), want.flatten(0, 1))
    assert torch.equal(f2, final)
    state, at = d["init"].clone(), 0
    for n in (64, 128, 0, 108):
        piece = {k: v[:, at:at + n] if k in ("u", "delta", "z", "B", "C") else v
                 for k, v in d.items()}
        piece["init"] = state
        assert torch.equal(call(canon, piece, final_state=state), want[:, at:at + n])
        at += n
    assert torch.equal(state, final)
    with canon.schedule(grid=3):
        assert torch.equal(call(canon, d), want)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,channels,groups,states", [(70, 40, 1, 16), (128, 17, 1, 7),
                                                         (1, 40, 2, 16), (67, 30, 2, 3)])
def test_many_sequences(canon, dtype, rows, channels, groups, states):
    """Enough sequences that each is walked whole: the forward bits of each
    alone (walked in chunks); gradients against the float64 form for some, the
    parameters' against the packed call's (walked in chunks)."""
    n = 460
    d = cuda(inputs(dtype, [rows] * n, channels, groups, states, False, rows))
    final = torch.empty_like(d["init"])
    keep = canon.selective_scan_states(d["u"], states)
    out = call(canon, d, final_state=final, states=keep)

    def grads(d, keep):
        return canon.selective_scan_grad(
            d["dout"], d["u"], d["delta"], d["A"], d["B"], d["C"], keep, D=d["D"], z=d["z"],
            delta_bias=d["bias"], delta_softplus=True, starts=d["starts"],
            d_final_state=d["dfinal"])

    got = grads(d, keep)
    per_seq = ("u", "delta", "z", "B", "C", "init", "dout", "dfinal")
    for i in (0, 201, 459):
        one = {k: v[i:i + 1].contiguous() if k in per_seq else v for k, v in d.items()}
        f = torch.empty_like(one["init"])
        assert torch.equal(call(canon, one, final_state=f), out[i:i + 1])
        assert torch.equal(f, final[i:i + 1])
        host = {k: v.cpu() if torch.is_tensor(v) else v for k, v in one.items()}
        names = ["u", "delta", "B", "C", "z", "init"]
        o, h, e = reference(host, leaves=names)
        want = torch.autograd.grad((o * e["dout"]).sum() + (h * e["dfinal"]).sum(),
                                   [e[k] for k in names])
        size = grad_sizes(host, True, names + ["A", "D", "bias"])
        mine = [got.du, got.ddelta, got.dB, got.dC, got.dz, got.dinit_state]
        for k, a, b in zip(names, mine, want):
            seq_ref.close(a[i:i + 1], b, size[k], 2 * terms(rows) + channels, (i, k))
    flat = ("u", "delta", "z", "B", "C", "dout")
    packed = {k: v.flatten(0, 1) if k in flat else v for k, v in d.items()}
    packed["starts"] = (torch.arange(n + 1) * rows).int().cuda()
    keep = canon.selective_scan_states(packed["u"], states, packed["starts"])
    assert torch.equal(call(canon, packed, states=keep), out.flatten(0, 1))
    other = grads(packed, keep)
    # each sum is within (2 terms + rows n) roundings of its absolute terms, of
    # which a value of n random ones is at least a 1 / sqrt(n rows) part
    bound = 2 * (2 * terms(rows) + 64) * seq_ref.U32 * (n * rows) ** 0.5
    for k in ("dA", "dD", "ddelta_bias"):
        a, b = getattr(got, k).double(), getattr(other, k).double()
        assert float((a - b).abs().max() / b.abs().max()) <= bound, k


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("channels,groups,states", [(1, 1, 1), (40, 2, 16), (65, 1, 8),
                                                    (96, 3, 13), (20, 1, 3), (130, 1, 4)])
def test_step(canon, dtype, channels, groups, states):
    d = inputs(dtype, [1] * 9, channels, groups, states, False, channels)
    g = cuda(d)
    row = {k: v[:, 0] if k in ("u", "delta", "z", "B", "C") else v for k, v in g.items()}
    for full in (True, False):
        kw = dict(D=row["D"], z=row["z"], delta_bias=row["bias"],
                  delta_softplus=True) if full else {}
        delta = row["delta"] if full else row["delta"].abs()
        state = g["init"].clone() if full else torch.zeros_like(g["init"])
        nxt = torch.full_like(state, 7.0)
        a = canon.selective_scan_step(state, row["u"], delta, row["A"], row["B"], row["C"],
                                      out_state=nxt, **kw)
        b = canon.selective_scan_step(state, row["u"], delta, row["A"], row["B"], row["C"], **kw)
        assert torch.equal(a, b) and torch.equal(state, nxt)
        out, h, _ = reference(d, full)
        size, hsize, _ = reference(d, full, absolute=True)
        seq_ref.close(a, out[:, 0], size[:, 0], terms(1), "out")
        seq_ref.close(state, h, hsize, terms(1), "state")


@pytest.mark.parametrize("channels,groups,states", [(40, 2, 16), (17, 1, 13), (64, 1, 8)])
def test_step_of_many_sequences(canon, channels, groups, states):
    """Enough sequences that a thread takes four: the bits of a few alone."""
    n = 8195
    d = cuda(inputs(BF16, [1] * n, channels, groups, states, False, channels))
    row = {k: v[:, 0] if k in ("u", "delta", "z", "B", "C") else v for k, v in d.items()}

    def go(at, state):
        return canon.selective_scan_step(state, row["u"][at], row["delta"][at], row["A"],
                                         row["B"][at], row["C"][at], D=row["D"], z=row["z"][at],
                                         delta_bias=row["bias"], delta_softplus=True)

    state = d["init"].clone()
    out = go(slice(None), state)
    for at in (slice(0, 9), slice(4095, 4100), slice(n - 3, n)):
        few = d["init"][at].clone()
        assert torch.equal(go(at, few), out[at]) and torch.equal(few, state[at])


def test_step_without_groups_dimension_and_strides(canon):
    d = cuda(inputs(BF16, [1] * 6, 48, 1, 16, False))
    big = torch.randn(6, 300, device="cuda").to(BF16)
    u, delta = big[:, 1:49], big[:, 50:98]
    B, C = big[:, 101:117], big[:, 120:136]
    z = big[:, 200:248]
    s1, s2 = d["init"].clone(), d["init"].clone()
    a = canon.selective_scan_step(s1, u, delta, d["A"], B, C, D=d["D"], z=z, delta_softplus=True)
    b = canon.selective_scan_step(s2, u.contiguous(), delta.contiguous(), d["A"],
                                  B.contiguous()[:, None], C.contiguous()[:, None], D=d["D"],
                                  z=z.contiguous(), delta_softplus=True)
    assert torch.equal(a, b) and torch.equal(s1, s2)


def test_strides_and_alignment(canon):
    """Slices of wider rows, no 16-byte alignment, interleaved sequences."""
    big = torch.randn(2, 70, 400, device="cuda").to(F16)
    A = -torch.rand(40, 16, device="cuda")
    v = dict(u=big[..., 1:41], delta=big[..., 43:83], z=big[..., 90:130], B=big[..., 131:147],
             C=big[..., 150:166])
    out = torch.full((2, 70, 50), 7.0, dtype=F16, device="cuda")

    def go(v, out=None):
        return canon.selective_scan(v["u"], v["delta"], A, v["B"], v["C"], z=v["z"],
                                    delta_softplus=True, out=out)

    want = go({k: t.contiguous() for k, t in v.items()})
    go(v, out[..., 3:43])
    assert torch.equal(out[..., 3:43], want)
    assert (out[..., :3] == 7).all() and (out[..., 43:] == 7).all()
    inter = {k: t.transpose(0, 1).contiguous().transpose(0, 1) for k, t in v.items()}
    assert torch.equal(go(inter), want)
    dout = torch.randn_like(want)
    keep = canon.selective_scan_states(v["u"], 16)
    canon.selective_scan(v["u"], v["delta"], A, v["B"], v["C"], z=v["z"], delta_softplus=True,
                         states=keep)
    g1 = canon.selective_scan_grad(dout, v["u"], v["delta"], A, v["B"], v["C"], keep, z=v["z"],
                                   delta_softplus=True)
    c = {k: t.contiguous() for k, t in v.items()}
    g2 = canon.selective_scan_grad(dout, c["u"], c["delta"], A, c["B"], c["C"], keep, z=c["z"],
                                   delta_softplus=True)
    for a, b in zip(g1, g2):
        assert (a is None and b is None) or torch.equal(a, b)
    e = v["u"][:1].expand(2, 70, 40)  # one row of inputs for both sequences
    assert torch.equal(go({**v, "u": e}), go({**v, "u": e.contiguous()}))


def test_rows_outside_sequences_and_special_values(canon):
    d = cuda(inputs(BF16, [200], 40, 1, 16, True, 8))
    d["starts"] = torch.tensor([3, 90, 90, 171]).int().cuda()
    d["init"] = torch.randn(3, 40, 16).cuda()
    out = torch.full((200, 40), 7.0, dtype=BF16, device="cuda")
    final = torch.full_like(d["init"], 7.0)
    call(canon, d, out=out, final_state=final)
    assert (out[:3] == 7).all() and (out[171:] == 7).all()
    assert torch.equal(final[1], d["init"][1])  # an empty sequence
    e = {k: v.clone() if torch.is_tensor(v) else v for k, v in d.items()}
    for k in ("u", "delta", "z", "B", "C"):
        e[k][:3], e[k][171:], e[k][90:171] = float("nan"), float("inf"), float("nan")
    got, f = torch.empty_like(out), torch.empty_like(final)
    call(canon, e, out=got, final_state=f)
    assert torch.equal(got[3:90], out[3:90]) and torch.equal(f[:2], final[:2])
    # a NaN in a row reaches that row and later ones of its channel alone
    e = {k: v.clone() if torch.is_tensor(v) else v for k, v in d.items()}
    e["u"][50, 7] = float("nan")
    got = call(canon, e)
    bad = torch.isnan(got[3:90])
    assert bad[47:, 7].all() and int(bad.sum()) == 40
    # steps so large that a is 0, and zero steps
    e = {k: v.clone() if torch.is_tensor(v) else v for k, v in d.items()}
    e["delta"].fill_(3e4)
    assert torch.isfinite(call(canon, e)[3:171].float()).all()
    e["delta"].fill_(float("-inf"))  # softplus 0: nothing decays, nothing is added
    call(canon, e, final_state=final)
    assert torch.equal(final, e["init"])
    # growing states: a zero one stays what the rows add, though exp(A sum dl)
    # over a chunk overflows
    e = {k: v.clone() if torch.is_tensor(v) else v for k, v in d.items()}
    e["A"] = e["A"].abs() * 0 + 40.0
    e["init"].zero_()
    e["u"].zero_()
    assert not call(canon, e, final_state=final)[3:171].any() and not final.any()
    # gradients: rows of other sequences do not count
    e = {k: v.clone() if torch.is_tensor(v) else v for k, v in d.items()}
    for k in ("u", "delta", "z", "B", "C", "dout"):
        e[k][:3], e[k][171:] = float("nan"), float("inf")
    res = []
    for x in (d, e):
        keep = canon.selective_scan_states(x["u"], 16, x["starts"])
        call(canon, x, states=keep)
        res.append(canon.selective_scan_grad(
            x["dout"], x["u"], x["delta"], x["A"], x["B"], x["C"], keep, D=x["D"], z=x["z"],
            delta_bias=x["bias"], delta_softplus=True, starts=x["starts"]))
    for name, a, b in zip(res[0]._fields, *res):
        if name in ("du", "ddelta", "dB", "dC", "dz"):
            a, b = a[3:171], b[3:171]
        assert torch.equal(a, b), name


def test_few_packed_rows_not_from_the_first(canon):
    """Few packed rows (each sequence walked whole), rows in front of and behind
    the sequences, empty ones between: as the sequences alone; the parameters'
    gradients take nothing from slots without rows."""
    d = cuda(inputs(F32, [120], 24, 1, 16, True, 4))
    d["starts"] = torch.tensor([7, 7, 70, 70, 70, 101]).int().cuda()
    d["init"] = torch.randn(5, 24, 16).cuda()
    names = ("u", "delta", "z", "B", "C", "dout")
    parts, total = [], 0
    for s, (a, b) in enumerate(((7, 7), (7, 70), (70, 70), (70, 70), (70, 101))):
        one = {k: v[None, a:b].contiguous() if k in names else v for k, v in d.items()}
        one["starts"], one["init"] = None, d["init"][s:s + 1]
        keep = canon.selective_scan_states(one["u"], 16)
        out = call(canon, one, states=keep)
        parts.append((out[0], canon.selective_scan_grad(
            one["dout"], one["u"], one["delta"], one["A"], one["B"], one["C"], keep, D=one["D"],
            z=one["z"], delta_bias=one["bias"], delta_softplus=True)))
    ws = torch.full((canon.selective_scan_grad_workspace_bytes(5, 120, True, 24, 1, 16),), 255,
                    dtype=torch.uint8, device="cuda")  # NaN wherever it is not written
    keep = canon.selective_scan_states(d["u"], 16, d["starts"])
    out = call(canon, d, states=keep)
    g = canon.selective_scan_grad(d["dout"], d["u"], d["delta"], d["A"], d["B"], d["C"], keep,
                                  D=d["D"], z=d["z"], delta_bias=d["bias"], delta_softplus=True,
                                  starts=d["starts"], ws=ws)
    assert torch.equal(out[7:101], torch.cat([p[0] for p in parts]))
    assert torch.equal(g.du[7:101], torch.cat([p[1].du[0] for p in parts]))
    assert torch.equal(g.dB[7:101], torch.cat([p[1].dB[0] for p in parts]))
    assert torch.equal(g.dinit_state, torch.cat([p[1].dinit_state for p in parts]))
    for k in ("dA", "dD", "ddelta_bias"):  # the same chunks' sums, in another order
        want = sum(getattr(p[1], k).double() for p in parts)
        got = getattr(g, k).double()
        assert float((got - want).abs().max() / want.abs().max()) <= 8 * seq_ref.U32, k


def test_empty(canon):
    d = cuda(inputs(F32, [5, 5], 24, 1, 16, False))
    for cut in ((slice(0, 0), slice(None)), (slice(None), slice(0, 0))):
        e = {k: v[cut] if k in ("u", "delta", "z", "B", "C", "dout") else v
             for k, v in d.items()}
        e["init"] = d["init"][cut[0]]
        final = torch.full_like(e["init"], 7.0)
        assert call(canon, e, final_state=final).shape == e["u"].shape
        assert torch.equal(final, e["init"])
        keep = canon.selective_scan_states(e["u"], 16)
        call(canon, e, states=keep)
        g = canon.selective_scan_grad(e["dout"], e["u"], e["delta"], e["A"], e["B"], e["C"], keep,
                                      D=e["D"], z=e["z"], delta_bias=e["bias"])
        assert not g.dA.any() and not g.dD.any() and not g.ddelta_bias.any()
        assert not g.dinit_state.any()


def test_refusals(canon):
    d = cuda(inputs(F32, [9, 9], 24, 1, 16, False))

    def go(**kw):
        a = {**d, **kw}
        return canon.selective_scan(a["u"], a["delta"], a["A"], a["B"], a["C"], D=a["D"],
                                    starts=a["starts"], init_state=a.get("st"))

    go()
    with pytest.raises(TypeError):
        go(u=d["u"].double())
    for bad in (dict(delta=d["delta"].half()), dict(delta=d["delta"][:, :8]),
                dict(A=d["A"].t()), dict(A=d["A"][:, ::2]), dict(B=d["B"][..., :8]),
                dict(B=torch.zeros(2, 9, 5, 16, device="cuda"),
                     C=torch.zeros(2, 9, 5, 16, device="cuda")),
                dict(D=d["D"].double()), dict(D=d["D"][:3]), dict(u=d["u"].cpu()),
                dict(st=d["init"][:1]), dict(u=d["u"].transpose(1, 2)),
                dict(starts=torch.tensor([0, 9], device="cuda").int()),
                dict(A=torch.zeros(24, 17, device="cuda"),
                     B=torch.zeros(2, 9, 1, 17, device="cuda"),
                     C=torch.zeros(2, 9, 1, 17, device="cuda"))):
        with pytest.raises(ValueError):
            go(**bad)
    with pytest.raises(ValueError):
        canon.selective_scan_step(d["init"], d["u"], d["delta"], d["A"], d["B"], d["C"])
    with pytest.raises(ValueError):
        canon.selective_scan_grad(d["dout"], d["u"], d["delta"], d["A"], d["B"], d["C"],
                                  torch.zeros(3, device="cuda"))


@pytest.mark.parametrize("lens,packed", [([17], False), ([100, 100], False), ([300], False),
                                         ([130, 9, 70], True)])
def test_states_that_keep_nothing(canon, lens, packed):
    """A of minus infinity, or beyond float32 once it is scaled: exp(dl A) is 0, so
    the state is the last row's alone.  Rows past a sequence's end inside a tile,
    whose step size is 0, change nothing."""
    d = inputs(F32, lens, 40, 1, 16, packed, 21)
    finite = dict(d, A=d["A"].clone())
    finite["A"][:, 3:9] = -1e30
    for low in (float("-inf"), -3.3e38):
        d["A"] = finite["A"].clone()
        d["A"][:, 3:9] = low
        g = cuda(d)
        final = torch.empty_like(g["init"])
        keep = canon.selective_scan_states(g["u"], 16, g["starts"])
        got = call(canon, g, final_state=final, states=keep)
        out, h, _ = reference(finite)
        size, hsize, _ = reference(finite, absolute=True)
        n = terms(max(lens))
        seq_ref.close(got, out, size, n, "out")
        seq_ref.close(final, h, hsize, n, "final")
        grads = canon.selective_scan_grad(
            g["dout"], g["u"], g["delta"], g["A"], g["B"], g["C"], keep, D=g["D"], z=g["z"],
            delta_bias=g["bias"], delta_softplus=True, starts=g["starts"])
        for name, t in zip(grads._fields, grads):
            assert torch.isfinite(t).all(), name
        assert not grads.dA[:, 3:9].any()
        step = torch.empty_like(final)
        one = {k: g[k].reshape(-1, *g[k].shape[1 if packed else 2:])[:len(lens)]
               for k in ("u", "delta", "z", "B", "C")}
        canon.selective_scan_step(g["init"], one["u"], one["delta"], g["A"], one["B"], one["C"],
                                  g["D"], one["z"], g["bias"], True, out_state=step)
        assert torch.isfinite(step).all()


def gradients(canon, d, keep, **kw):
    return canon.selective_scan_grad(
        d["dout"], d["u"], d["delta"], d["A"], d["B"], d["C"], keep, D=d["D"], z=d["z"],
        delta_bias=d["bias"], delta_softplus=True, starts=d["starts"], d_final_state=d["dfinal"],
        **kw)


FIELDS = dict(u="du", delta="ddelta", A="dA", B="dB", C="dC", D="dD", z="dz", bias="ddelta_bias",
              init="dinit_state")
PARAMS = ("A", "D", "bias")


def check_gradients(got, want, size, rows, chunks, what, names=tuple(FIELDS), at=slice(None)):
    """rows: of a sequence; chunks: of all.  A parameter's gradient adds at most 64
    rows of a chunk, then a 16th of the chunks, then 16 lanes; dB and dC add a
    group's channels, 16 lanes by folding, then waves and slabs (below 64)."""
    for k in names:
        extra = 64 + chunks / 16 + 8 if k in PARAMS else 64
        g = getattr(got, FIELDS[k])
        seq_ref.close(g if k in PARAMS else g[at], want[k].cpu(), size[k].cpu(),
                      2 * terms(rows) + extra, (what, k))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("n,rows,channels,groups,states", [
    (400, 200, 24, 1, 16), (400, 257, 24, 1, 5), (256, 193, 24, 2, 3), (170, 129, 130, 1, 16)])
def test_whole_sequences_of_many_chunks(canon, dtype, n, rows, channels, groups, states):
    """Enough sequences of three chunks or more that a wave walks each whole, both
    ways: the forward bits of each alone (in chunks), the gradients against the
    float64 formulas; with the incoming gradient of one sequence alone the
    parameters' gradients are that sequence's, every chunk of it."""
    chunks = -(-rows // 64)
    d = cuda(inputs(dtype, [rows] * n, channels, groups, states, False, rows + n))
    # sums of one sign, so that no part of them is lost in the bound
    for k in ("u", "B", "C", "D", "z", "dout", "init", "dfinal"):
        d[k] = d[k].abs()
    final, keep = torch.empty_like(d["init"]), canon.selective_scan_states(d["u"], states)
    assert launches(lambda: call(canon, d)) == 1
    out = call(canon, d, final_state=final, states=keep)
    per = ("u", "delta", "z", "B", "C", "init", "dout", "dfinal")
    for i in (0, n // 2 + 1, n - 1):
        one = {k: v[i:i + 1].contiguous() if k in per else v for k, v in d.items()}
        f, k1 = torch.empty_like(one["init"]), canon.selective_scan_states(one["u"], states)
        assert launches(lambda: call(canon, one)) == 3
        assert torch.equal(call(canon, one, final_state=f, states=k1), out[i:i + 1])
        assert torch.equal(f, final[i:i + 1])
        saved = -(-rows // 16)  # every 16 rows, of 4 places a chunk
        assert torch.equal(k1.view(4 * chunks, -1)[:saved],
                           keep.view(n, 4 * chunks, -1)[i, :saved])
    assert launches(lambda: gradients(canon, d, keep)) == 2
    got = gradients(canon, d, keep)
    o, h, want = seq_ref.scan_grads(d)
    so, sh, size = seq_ref.scan_grads(d, absolute=True)
    seq_ref.close(out, o.cpu(), so.cpu(), terms(rows), "out")
    seq_ref.close(final, h.cpu(), sh.cpu(), terms(rows), "final")
    check_gradients(got, want, size, rows, n * chunks, "all")
    for i in (0, n // 2 + 1, n - 1):
        e = dict(d, dout=torch.zeros_like(d["dout"]), dfinal=torch.zeros_like(d["dfinal"]))
        e["dout"][i], e["dfinal"][i] = d["dout"][i], d["dfinal"][i]
        got = gradients(canon, e, keep)
        one = {k: v[i:i + 1] if k in per else v for k, v in d.items()}
        _, _, want = seq_ref.scan_grads(one)
        _, _, size = seq_ref.scan_grads(one, absolute=True)
        check_gradients(got, want, size, rows, chunks, i, at=slice(i, i + 1))
        others = torch.arange(n, device="cuda") != i
        assert not got.du[others].any() and not got.dinit_state[others].any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,channels,groups,states", [
    (1024, 40, 1, 16), (1025, 17, 1, 3), (2117, 20, 2, 7), (3100, 8, 1, 16)])
def test_carries_of_many_chunks(canon, dtype, rows, channels, groups, states):
    """16 chunks and more of one sequence, whose carries pass between the chunks
    in batches of 16, both ways: forward the bits of pieces of one chunk, backward
    the float64 formulas."""
    d = cuda(inputs(dtype, [rows], channels, groups, states, False, rows))
    d["bias"] -= 2.0  # smaller steps, so that states live through many chunks
    for k in ("u", "B", "C", "D", "z", "dout", "init", "dfinal"):
        d[k] = d[k].abs()
    final, keep = torch.empty_like(d["init"]), canon.selective_scan_states(d["u"], states)
    assert launches(lambda: call(canon, d)) == 3
    out = call(canon, d, final_state=final, states=keep)
    state = d["init"].clone()
    for at in range(0, rows, 64):
        piece = {k: v[:, at:at + 64] if k in ("u", "delta", "z", "B", "C") else v
                 for k, v in d.items()}
        piece["init"] = state
        assert torch.equal(call(canon, piece, final_state=state), out[:, at:at + 64]), at
    assert torch.equal(state, final)
    assert launches(lambda: gradients(canon, d, keep)) == 4
    got = gradients(canon, d, keep)
    _, _, want = seq_ref.scan_grads(d)
    _, _, size = seq_ref.scan_grads(d, absolute=True)
    check_gradients(got, want, size, rows, -(-rows // 64), "alone")
    # packed behind and before others: the same bits, those of parameters aside
    lens = [70, rows, 0, 1100]
    p = cuda(inputs(dtype, lens, channels, groups, states, True, 3))
    p.update({k: d[k] for k in ("A", "D", "bias")})
    for k in ("u", "delta", "z", "B", "C", "dout"):
        p[k][70:70 + rows] = d[k][0]
    p["init"][1], p["dfinal"][1] = d["init"][0], d["dfinal"][0]
    f2, keep = torch.empty_like(p["init"]), canon.selective_scan_states(p["u"], states, p["starts"])
    assert torch.equal(call(canon, p, final_state=f2, states=keep)[70:70 + rows], out[0])
    assert torch.equal(f2[1], final[0])
    other = gradients(canon, p, keep)
    for k in ("du", "ddelta", "dB", "dC", "dz"):
        assert torch.equal(getattr(other, k)[70:70 + rows], getattr(got, k)[0]), k
    assert torch.equal(other.dinit_state[1], got.dinit_state[0])
