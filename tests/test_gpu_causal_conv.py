"""Causal convolution against its float64 form: forward, backward, single rows."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import seq_ref  # noqa: E402

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def canon():
    import scan_canonical_reduce_amd as c
    return c


def inputs(dtype, lens, channels, taps, packed, seed=0, param=F32):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g)

    lead = (sum(lens),) if packed else (len(lens), lens[0])
    starts = torch.tensor([0] + lens).cumsum(0).int() if packed else None
    return dict(x=normal(*lead, channels).to(dtype), w=normal(channels, taps).to(param),
                b=normal(channels).to(param), init=normal(len(lens), taps - 1, channels).to(dtype),
                dout=normal(*lead, channels).to(dtype),
                dfinal=normal(len(lens), taps - 1, channels).to(dtype), starts=starts)


def cuda(d):
    return {k: v.cuda() if torch.is_tensor(v) else v for k, v in d.items()}


def reference(d, act, bias=True, init=True, grad=False):
    """float64 values, and the sums of absolute terms behind them."""
    x, w = d["x"].double(), d["w"].double()
    b = d["b"].double() if bias else None
    st = d["init"].double() if init else torch.zeros_like(d["init"]).double()
    leaves = [t.requires_grad_() for t in (x, w, st)] + ([b.requires_grad_()] if bias else [])
    outs, sizes, finals = [], [], []
    for i, at in enumerate(seq_ref.spans(d["x"], d["starts"])):
        y, f = seq_ref.conv_one(x[at], w, b, act, st[i])
        s, _ = seq_ref.conv_one(x[at].abs(), w.abs(), None if b is None else b.abs(), False,
                                st[i].abs())
        outs.append(y), sizes.append(s), finals.append(f)
    join = torch.stack if d["starts"] is None else torch.cat
    out, size, final = join(outs), join(sizes), torch.stack(finals)
    if not grad:
        return out, size, final
    loss = (out * d["dout"].double()).sum() + (final * d["dfinal"].double()).sum()
    return out, torch.autograd.grad(loss, leaves)


# p adds taps + 1 terms in FMAs (one rounding each); silu multiplies by a
# sigmoid with a relative error below 8 roundings, whose argument's error is
# at most the error of p (slope of p sigmoid(p) below 1.1): 2 (taps + 2) + 12
# roundings of the absolute sum cover both.
def terms(taps):
    return 2 * (taps + 2) + 12


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("taps", [1, 2, 3, 4, 8])
@pytest.mark.parametrize("channels", [1, 24, 37, 264])
@pytest.mark.parametrize("act", [None, "silu"])
def test_forward(canon, dtype, taps, channels, act):
    for packed, lens in ((False, [1, 1]), (False, [33, 33, 33]),
                         (True, [5, 0, 64, 1, 31, 0, 2, 100])):
        d = inputs(dtype, lens, channels, taps, packed, taps + channels)
        g = cuda(d)
        final = torch.empty_like(g["init"])
        got = canon.causal_conv(g["x"], g["w"], g["b"], act, g["starts"], g["init"], final)
        out, size, last = reference(d, act)
        seq_ref.close(got, out, size, terms(taps), (lens, packed))
        assert torch.equal(final.cpu().double(), last)
        got = canon.causal_conv(g["x"], g["w"], None, act, g["starts"])
        out, size, _ = reference(d, act, bias=False, init=False)
        seq_ref.close(got, out, size, terms(taps), (lens, packed, "plain"))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_long_runs(canon, dtype):
    """Enough rows for the long-run variant, which must give the same bits as
    the short one on each sequence alone."""
    d = cuda(inputs(dtype, [1040] * 8, 4096, 4, False))
    got = canon.causal_conv(d["x"], d["w"], d["b"], "silu", None, d["init"])
    one = canon.causal_conv(d["x"][2:3, :100], d["w"], d["b"], "silu", None,
                            d["init"][2:3].contiguous())
    assert torch.equal(got[2:3, :100], one)
    tail = canon.causal_conv(d["x"][5:6, 900:], d["w"], d["b"], "silu", None,
                             d["x"][5:6, 897:900].contiguous())
    assert torch.equal(got[5:6, 900:], tail)


def test_parameters_of_the_activation_type(canon):
    d = inputs(BF16, [50], 48, 4, False, param=BF16)
    g = cuda(d)
    got = canon.causal_conv(g["x"], g["w"], g["b"], "silu", None, g["init"])
    out, size, _ = reference(d, "silu")
    seq_ref.close(got, out, size, terms(4))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("taps", [1, 2, 4, 7])
@pytest.mark.parametrize("channels", [24, 37])
@pytest.mark.parametrize("act", [None, "silu"])
def test_backward(canon, dtype, taps, channels, act):
    for packed, lens in ((False, [1]), (False, [70, 70]), (True, [3, 0, 65, 1, 32, 2, 0])):
        d = inputs(dtype, lens, channels, taps, packed, 7 * taps + channels)
        g = cuda(d)
        got = canon.causal_conv_grad(g["dout"], g["x"], g["w"], g["b"], act, g["starts"],
                                     g["init"], g["dfinal"])
        _, (dx, dw, dst, db) = reference(d, act, grad=True)
        # Sums of absolute terms: |silu'| <= 1.1, and p's relative error enters
        # through silu'' <= 0.5 times the absolute sum of p (at most ~ 6 taps
        # here): the bounds below use 1.1 + that.
        w = d["w"].double().abs()
        _, psize, _ = reference(d, None)
        psize = float(psize.detach().max()) if psize.numel() else 0.0
        gmax = 1.1 + psize
        gout = d["dout"].double().abs().max() if d["dout"].numel() else 0.0
        big = float(gout) * gmax
        size = (w.sum(1) * big + float(d["dfinal"].abs().max() if taps > 1 else 0)).expand_as(dx)
        n = 2 * terms(taps)
        seq_ref.close(got.dx, dx, size, n, (lens, "dx"))
        rows = sum(lens)
        seq_ref.close(got.dweight, dw, torch.full_like(dw, rows * big * 5), n + 64, (lens, "dw"))
        seq_ref.close(got.dbias, db, torch.full_like(db, rows * big), n + 64, (lens, "db"))
        seq_ref.close(got.dinit_state, dst, size.max().expand_as(dst) if dst.numel() else dst, n,
                      (lens, "dinit"))


def test_backward_against_differences(canon):
    """<gradient, v> against a central difference of the float64 form along v:
    with step 1e-5 its error is about 1e-10 |f'''| + 1e-11 |f|."""
    d = inputs(F32, [40, 0, 7], 24, 4, True)
    g = cuda(d)
    got = canon.causal_conv_grad(g["dout"], g["x"], g["w"], g["b"], "silu", g["starts"],
                                 g["init"], g["dfinal"])
    for key, grad in (("x", got.dx), ("w", got.dweight), ("b", got.dbias),
                      ("init", got.dinit_state)):
        v = torch.randn(d[key].shape, generator=torch.Generator().manual_seed(1)).double()

        def f(step):
            e = {k: t.double() if torch.is_tensor(t) and t.is_floating_point() else t
                 for k, t in d.items()}
            e[key] = e[key] + step * v
            out, _, final = reference(e, "silu")
            return float(((out * e["dout"]).sum() + (final * e["dfinal"]).sum()).detach())

        want = (f(1e-5) - f(-1e-5)) / 2e-5
        assert float((grad.double().cpu() * v).sum()) == pytest.approx(want, rel=1e-5, abs=1e-4)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("taps", [1, 3, 4])
@pytest.mark.parametrize("channels", [37, 48])
def test_step_equals_the_sequence(canon, dtype, taps, channels):
    """Row after row, the step gives the sequence's bits, in place or not."""
    d = cuda(inputs(dtype, [9] * 5, channels, taps, False))
    final = torch.empty_like(d["init"])
    want = canon.causal_conv(d["x"], d["w"], d["b"], "silu", None, d["init"], final)
    state, other = d["init"].clone(), d["init"].clone()
    for t in range(9):
        nxt = torch.empty_like(other)
        a = canon.causal_conv_step(d["x"][:, t], state, d["w"], d["b"], "silu")
        b = canon.causal_conv_step(d["x"][:, t], other, d["w"], d["b"], "silu", out_state=nxt)
        other = nxt
        assert torch.equal(a, want[:, t]) and torch.equal(b, want[:, t])
        assert torch.equal(state, other)
    assert torch.equal(state, final)


def test_state_in_place_and_pieces(canon):
    """A sequence in pieces, the state handed on in one buffer: the same bits."""
    d = cuda(inputs(BF16, [77] * 3, 64, 4, False))
    want = canon.causal_conv(d["x"], d["w"], d["b"], "silu", None, d["init"])
    state = d["init"].clone()
    at = 0
    for n in (1, 2, 40, 0, 34):
        got = canon.causal_conv(d["x"][:, at:at + n], d["w"], d["b"], "silu", None, state, state)
        assert torch.equal(got, want[:, at:at + n])
        at += n
    assert torch.equal(state, d["x"][:, 74:])


def test_rows_outside_sequences_and_strides(canon):
    x = torch.randn(50, 130).to(BF16).cuda()
    w, b = torch.randn(64, 4).cuda(), torch.randn(64).cuda()
    starts = torch.tensor([3, 20, 20, 41], dtype=torch.int32).cuda()
    out = torch.full((50, 70), 7.0, dtype=BF16, device="cuda")
    canon.causal_conv(x[:, 2:66], w, b, "silu", starts, out=out[:, 4:68])
    want = canon.causal_conv(x[3:41, 2:66].contiguous(), w, b, "silu",
                             (starts - 3).int())
    assert torch.equal(out[3:41, 4:68], want)
    assert (out[:3] == 7).all() and (out[41:] == 7).all() and (out[:, :4] == 7).all()
    # NaN behind the sequences and in the next sequence reach nothing
    y = x.clone()
    y[41:], y[:3], y[20:41] = float("nan"), float("inf"), float("nan")
    got = canon.causal_conv(y[:, 2:66], w, b, "silu", starts)
    assert torch.equal(got[3:20], want[:17])
    # interleaved sequences: [rows, sequences, channels] transposed
    z = torch.randn(30, 2, 64).cuda()
    got = canon.causal_conv(z.transpose(0, 1), w, b)
    assert torch.equal(got, canon.causal_conv(z.transpose(0, 1).contiguous(), w, b))
    g1 = canon.causal_conv_grad(x[:, 2:66], x[:, 66:130], w, b, "silu", starts)
    y = x.clone()
    y[:3], y[41:] = float("nan"), float("inf")
    g2 = canon.causal_conv_grad(y[:, 2:66], y[:, 66:130], w, b, "silu", starts)
    assert torch.equal(g1.dweight, g2.dweight) and torch.equal(g1.dbias, g2.dbias)
    assert torch.equal(g1.dx[3:41], g2.dx[3:41])


def test_broadcast_input_and_empty(canon):
    w, b = torch.randn(8, 4).cuda(), torch.randn(8).cuda()
    x = torch.randn(1, 20, 8).cuda()
    got = canon.causal_conv(x.expand(3, 20, 8), w, b)
    assert torch.equal(got[2], got[0])
    assert torch.equal(got[:1], canon.causal_conv(x, w, b))
    assert canon.causal_conv(x[:, :0], w, b).shape == (1, 0, 8)
    assert canon.causal_conv(x[:0], w, b).shape == (0, 20, 8)
    g = canon.causal_conv_grad(x[:, :0], x[:, :0], w, b)
    assert not g.dweight.any() and not g.dbias.any()
    g = canon.causal_conv_grad(x[:0], x[:0], w, b)
    assert not g.dweight.any() and not g.dbias.any()


def test_refusals(canon):
    x, w = torch.randn(2, 9, 8).cuda(), torch.randn(8, 4).cuda()
    with pytest.raises(TypeError):
        canon.causal_conv(x.double(), w)
    with pytest.raises(TypeError):
        canon.causal_conv(x, w.half())
    with pytest.raises(ValueError):
        canon.causal_conv(x, w, activation="relu")
    with pytest.raises(ValueError):
        canon.causal_conv(x, torch.randn(8, 9).cuda())  # too many taps
    with pytest.raises(ValueError):
        canon.causal_conv(x, w[:7])
    with pytest.raises(ValueError):
        canon.causal_conv(x[0], w)
    with pytest.raises(ValueError):
        canon.causal_conv(x, w, starts=torch.tensor([0, 9]).int().cuda())
    with pytest.raises(ValueError):
        canon.causal_conv(x[0], w, starts=torch.tensor([0, 9]).cuda())  # 64-bit
    with pytest.raises(ValueError):
        canon.causal_conv(x.transpose(1, 2), w[:, :4])
    with pytest.raises(ValueError):
        canon.causal_conv(x, w, init_state=torch.zeros(2, 4, 8).cuda())
    with pytest.raises(ValueError):
        canon.causal_conv(x, w, out=torch.empty(1, 9, 8).cuda().expand(2, 9, 8))
    with pytest.raises(ValueError):
        canon.causal_conv(x.cpu(), w)
    with pytest.raises(ValueError):
        canon.causal_conv_step(x, torch.zeros(2, 3, 8).cuda(), w)


@pytest.mark.parametrize("taps", [2, 3, 4, 8])
@pytest.mark.parametrize("rows", [64, 65, 66, 67, 68, 71, 72, 97])
def test_backward_near_the_end(canon, taps, rows):
    """A sequence that ends a few rows behind a run's: the gradients of the whole
    are those of the same rows in a longer buffer, whatever comes after them."""
    d = cuda(inputs(F32, [rows], 64, taps, False, seed=rows))
    want = canon.causal_conv_grad(d["dout"], d["x"], d["w"], d["b"], "silu")
    x, dout = (torch.full((2, rows + 8, 64), float("nan"), device="cuda") for _ in range(2))
    x[:, :rows], dout[:, :rows] = d["x"], d["dout"]
    got = canon.causal_conv_grad(dout[:1, :rows], x[:1, :rows], d["w"], d["b"], "silu")
    assert torch.equal(got.dx, want.dx) and torch.equal(got.dweight, want.dweight)
    e = {k: v.double().cpu() if torch.is_tensor(v) else v for k, v in d.items()}
    e["init"].zero_()
    e["dfinal"].zero_()
    _, (dx, dw, _, db) = reference(e, "silu", grad=True)
    # dp = dout silu'(p), with the slope of silu' below 1/2 and |silu'| < 1.1: p is
    # off by taps + 2 roundings of its absolute sum, the rest of dp by 20; then a
    # sum of `taps` (dx) or `rows` terms, in FMAs
    half = 2.0**-24
    xm, gm, wm, bm = (float(d[k].abs().max()) for k in ("x", "dout", "w", "b"))
    dp = gm * half * (0.5 * (taps + 2) * (bm + taps * wm * xm) + 20)
    tol = taps * wm * (dp + (taps + 1) * half * 1.1 * gm)
    assert (want.dx.double().cpu() - dx).abs().max() <= tol
    tol = rows * (dp + (rows + 2) * half * 1.1 * gm)
    assert (want.dweight.double().cpu() - dw).abs().max() <= tol * xm
    assert (want.dbias.double().cpu() - db).abs().max() <= tol


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("channels", [1, 2, 3, 4, 5, 6, 7, 9, 255, 1001])
def test_channels_of_any_number_and_place(canon, dtype, channels):
    """Channels that are not whole vectors, or not aligned to them: the bits of the
    same channels among more, states updated in place, nothing written beside."""
    wide, taps, rows, seqs = (channels + 15) // 8 * 8, 4, 77, 3
    d = cuda(inputs(dtype, [rows] * seqs, wide, taps, False, seed=channels))
    for off in (0, 1):
        cut = slice(off, off + channels)

        def own(t, dim=-1):  # the channels alone, contiguous
            return t.narrow(dim, off, channels).contiguous()

        w, b, init = own(d["w"], 0), own(d["b"]), own(d["init"])
        final = torch.empty_like(d["init"])
        want = canon.causal_conv(d["x"], d["w"], d["b"], "silu", None, d["init"], final)
        state = init.clone()
        out = torch.full_like(want, 7.0)
        canon.causal_conv(d["x"][..., cut], w, b, "silu", None, state, state, out[..., cut])
        assert torch.equal(out[..., cut], want[..., cut]) and torch.equal(state, own(final))
        assert (out[..., :off] == 7).all() and (out[..., off + channels:] == 7).all()
        g = canon.causal_conv_grad(d["dout"], d["x"], d["w"], d["b"], "silu", None, d["init"],
                                   d["dfinal"])
        dx = torch.full_like(want, 7.0)
        h = canon.causal_conv_grad(d["dout"][..., cut], d["x"][..., cut], w, b, "silu", None,
                                   init, own(d["dfinal"]), dx[..., cut])
        assert torch.equal(dx[..., cut], g.dx[..., cut])
        assert (dx[..., :off] == 7).all() and (dx[..., off + channels:] == 7).all()
        assert torch.equal(h.dweight, own(g.dweight, 0)) and torch.equal(h.dbias, own(g.dbias))
        assert torch.equal(h.dinit_state, own(g.dinit_state))
        all_state, state = d["init"].clone(), init.clone()
        for t in range(3):
            a = canon.causal_conv_step(d["x"][:, t], all_state, d["w"], d["b"], "silu")
            out = torch.full((seqs, channels + 5), 7.0, dtype=dtype, device="cuda")
            canon.causal_conv_step(d["x"][:, t, cut], state, w, b, "silu", out=out[:, :channels])
            assert torch.equal(out[:, :channels], a[:, cut]) and (out[:, channels:] == 7).all()
            assert torch.equal(state, own(all_state))


def inner_waves(rows, channels, taps, per):
    """Waves of the backward pass over one sequence of `rows` rows, `per` channels a
    lane, that run the loop without checks: every lane's run of 32 rows is full, is
    not the first, and has all the rows that whole fetches of 4 read."""
    read = (32 + taps - 1 + 3) // 4 * 4
    lanes = [32 * (i // -(-channels // per)) for i in range(-(-rows // 32) * -(-channels // per))]
    inner = [r > 0 and r + 32 <= rows and r + read <= rows for r in lanes]
    return sum(all(inner[i:i + 64]) for i in range(0, len(inner), 64))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("taps", [1, 2, 3, 4, 5, 8])
@pytest.mark.parametrize("channels", [128, 133])
def test_backward_without_checks(canon, dtype, taps, channels):
    """Sequences whose ends lie on both sides of the rows that the loop without
    checks needs, against the float64 form; NaN behind each sequence."""
    per = 2 if channels == 128 else 1
    need = 32 + (32 + taps - 1 + 3) // 4 * 4
    if channels == 128:
        assert not inner_waves(need - 1, channels, taps, per)
        assert inner_waves(need, channels, taps, per)
    assert inner_waves(230, channels, taps, per)
    for rows in (need - 1, need, need + 1, 230):
        d = inputs(dtype, [rows], channels, taps, False, seed=rows + taps)
        d["init"].zero_()
        d["dfinal"].zero_()
        g = cuda(d)
        x, dout = (torch.full((1, rows + 8, channels), float("nan"), dtype=dtype, device="cuda")
                   for _ in range(2))
        x[:, :rows], dout[:, :rows] = g["x"], g["dout"]
        dx = torch.full_like(x, 7.0)
        got = canon.causal_conv_grad(dout[:, :rows], x[:, :rows], g["w"], g["b"], "silu",
                                     dx=dx[:, :rows])
        assert (dx[:, rows:] == 7).all()
        _, (want, dw, _, db) = reference(d, "silu", grad=True)
        # With h = 2^-24 and pm the largest absolute sum of p: p is off by (taps + 2)
        # h pm, and silu' has a slope below 1/2.  silu' = q + p (q - q q), q off by
        # (1 - q) (2 |p| + 2) h + 3 h of itself, is off by 5 |p| h + 8 h more
        # (p^2 q (1 - q) < 1/2); the product with dout by 2 h.  Then a sum of `taps`
        # (dx) or `rows` terms of at most 1.1 gm, in FMAs.
        h = 2.0**-24
        xm, gm, wm, bm = (float(d[k].double().abs().max()) for k in ("x", "dout", "w", "b"))
        pm = bm + taps * wm * xm
        dp = gm * h * ((0.5 * (taps + 2) + 5) * pm + 10)
        tol = taps * wm * (dp + (taps + 1) * h * 1.1 * gm)
        err = (got.dx.double().cpu() - want).abs()
        assert (err <= tol + seq_ref.half_step(dtype) * (want.abs() + tol)).all(), rows
        tol = rows * (dp + (rows + 2) * h * 1.1 * gm)
        assert (got.dweight.double().cpu() - dw).abs().max() <= tol * xm, rows
        assert (got.dbias.double().cpu() - db).abs().max() <= tol, rows
    # packed, sequences of other lengths around, none starting with a run's start
    lens = [9, 0, 150, 31, need]
    d = inputs(dtype, lens, channels, taps, True, seed=taps)
    g = cuda(d)
    got = canon.causal_conv_grad(g["dout"], g["x"], g["w"], g["b"], "silu", g["starts"], g["init"],
                                 g["dfinal"])
    for s, (a, b) in enumerate(zip(d["starts"][:-1].tolist(), d["starts"][1:].tolist())):
        one = canon.causal_conv_grad(g["dout"][None, a:b], g["x"][None, a:b], g["w"], g["b"],
                                     "silu", None, g["init"][s:s + 1], g["dfinal"][s:s + 1])
        assert torch.equal(got.dx[a:b], one.dx[0])
        assert torch.equal(got.dinit_state[s], one.dinit_state[0])


def column_sum(parts, numbers):
    """parts[i] under the number numbers[i]: 16 lanes, each in order, then the
    pairwise tree over the lanes; float32."""
    lanes = [np.zeros_like(parts[0]) for _ in range(16)]
    for i, p in sorted(zip(numbers, parts), key=lambda x: x[0]):
        lanes[i % 16] = lanes[i % 16] + p
    while len(lanes) > 1:
        lanes = [a + b for a, b in zip(lanes[::2], lanes[1::2])]
    return lanes[0]


@pytest.mark.parametrize("starts", [
    None, [0, 32, 64], [0, 200, 200, 231, 600], [7, 7, 40, 41, 1000, 1640],
    list(range(3, 2400, 47))])
def test_parameter_sums_in_the_stated_order(canon, starts):
    """dweight and dbias bit for bit in the order that canon_seq.h states: of packed
    sequences by the numbers that starts gives the chunks.  The products of bfloat16
    values are exact in float32, and a float32 plus one is exact in float64, so each
    FMA is that sum rounded once."""
    channels, taps = 6, 3
    rows = 165 if starts is None else starts[-1] + 9
    lead = (5, rows) if starts is None else (rows,)
    g = torch.Generator().manual_seed(rows)
    x, dout = (torch.randn(*lead, channels, generator=g).to(BF16) for _ in range(2))
    w = torch.randn(channels, taps, generator=g)
    got = canon.causal_conv_grad(
        dout.cuda(), x.cuda(), w.cuda(), torch.zeros(channels).cuda(), None,
        None if starts is None else torch.tensor(starts, dtype=torch.int32).cuda())
    if starts is None:
        seqs = [(x[s], dout[s], s * -(-rows // 32)) for s in range(5)]
    else:
        seqs = [(x[a:b], dout[a:b], s + a // 32)
                for s, (a, b) in enumerate(zip(starts[:-1], starts[1:]))]
    dw, db, numbers = [], [], []
    for xs, ds, first in seqs:
        full = np.concatenate([np.zeros((taps - 1, channels)), xs.double().numpy()])
        ds = ds.double().numpy()
        for c in range(-(-len(ds) // 32)):
            w1, b1 = np.zeros((channels, taps), np.float32), np.zeros(channels, np.float32)
            for t in range(32 * c, min(32 * c + 32, len(ds))):
                b1 = (b1 + ds[t]).astype(np.float32)
                w1 = (w1 + full[t:t + taps].T * ds[t][:, None]).astype(np.float32)
            dw.append(w1), db.append(b1), numbers.append(first + c)
    assert np.array_equal(got.dbias.cpu().numpy(), column_sum(db, numbers))
    assert np.array_equal(got.dweight.cpu().numpy(), column_sum(dw, numbers))
    if starts is not None and len(starts) > 3:  # the order shows in the bits
        assert not np.array_equal(got.dweight.cpu().numpy(), column_sum(dw, range(len(dw))))
