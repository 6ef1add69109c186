"""Sampling against a sort in 80-bit numbers, token by token."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import layer_ref  # noqa: E402

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
INF = math.inf


@pytest.fixture(scope="module")
def canon():
    import scan_canonical_reduce_amd as c
    return c


def logits(dtype, rows, vocab, seed=0, scale=3.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, vocab, generator=g) * scale).to(dtype), torch.rand(rows, generator=g)


def expect(x, u, **settings):
    """Reference tokens, and which rows lie further from every border than the
    kernel's rounding can reach.  A weight is off by 2^-51 relative and half a step of
    2^-(62 - log2 vocab), so sums by less than 2^-50 + vocab 2^-62 2^log2 vocab of the
    largest weight: 2^-27 of the whole at most at 2^17 tokens, 2^-36 at 2^13."""
    rows, vocab = x.shape
    x = x.float().numpy()
    ids, sure = [], []
    for i in range(rows):
        s = {k: float(v[i]) if torch.is_tensor(v) else v for k, v in settings.items()}
        if "top_k" in s:
            s["top_k"] = int(s["top_k"])
        t, margin = layer_ref.sample(x[i], float(u[i]), **s)
        ids.append(t)
        sure.append(margin > 2.0 ** -50 + 4.0 * vocab * vocab * 2.0 ** -62)
    return torch.tensor(ids), torch.tensor(sure)


def check(canon, x, u, **settings):
    on = {k: v.cuda() if torch.is_tensor(v) else v for k, v in settings.items()}
    got = canon.sample(x.cuda(), u.cuda(), **on)
    want, sure = expect(x, u, **settings)
    assert sure.float().mean() > 0.9 or sure.numel() < 20
    bad = (got.cpu() != want) & sure
    assert not bad.any(), (settings, torch.nonzero(bad)[:4].tolist(), got.cpu()[bad][:4], want[bad][:4])
    return got


SETTINGS = [dict(), dict(temperature=0.7), dict(temperature=0.0), dict(top_k=1), dict(top_k=7),
            dict(top_p=0.9), dict(top_p=0.0), dict(min_p=0.1), dict(min_p=1.0),
            dict(temperature=1.3, top_k=20, top_p=0.8), dict(temperature=0.5, top_p=0.95, min_p=0.02),
            dict(top_k=5, min_p=0.3), dict(temperature=25.0, top_k=400, top_p=0.5, min_p=1e-3),
            dict(temperature=1e-6, top_p=0.9), dict(temperature=INF, top_k=100)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("vocab", [1, 2, 63, 64, 65, 100, 1000, 4096, 10007])
def test_settings(canon, dtype, vocab):
    for i, s in enumerate(SETTINGS):
        check(canon, *logits(dtype, 24, vocab, seed=i), **s)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("vocab", [32000, 50021, 131072])
def test_large_vocabularies(canon, dtype, vocab):
    for i, s in enumerate([dict(), dict(temperature=0.8, top_k=50, top_p=0.95),
                           dict(top_p=0.9), dict(top_k=5000, min_p=0.01),
                           dict(temperature=3.0, top_p=0.99)]):
        check(canon, *logits(dtype, 6, vocab, seed=i), **s)


def test_a_very_large_vocabulary(canon):
    for dtype in (F32, BF16):
        x, u = logits(dtype, 2, 700001, seed=1)
        for s in (dict(), dict(top_p=0.9), dict(top_k=50)):
            check(canon, x, u, **s)


@pytest.mark.parametrize("rows", [1, 2, 255, 700])
def test_rows(canon, rows):
    """Settings of their own for each row, few rows and many."""
    x, u = logits(BF16, rows, 1500, seed=rows)
    g = torch.Generator().manual_seed(rows)

    def pick(values, dt=F32):
        return torch.tensor(values, dtype=dt)[torch.randint(len(values), (rows,), generator=g)]

    check(canon, x, u, temperature=pick([0.0, 0.3, 1.0, 2.0, -1.0]),
          top_k=pick([0, 0, 1, 10, 5000, -3], torch.int32), top_p=pick([1.0, 0.5, 0.9, 2.0]),
          min_p=pick([0.0, 0.05, 0.5, 7.0, -1.0]))


@pytest.mark.parametrize("vocab", [8, 3000])
def test_masks(canon, vocab):
    """Minus infinity, NaN and the type's lowest value; rows of nothing else."""
    for dtype in (F32, BF16, F16):
        x, u = logits(dtype, 30, vocab, seed=vocab)
        g = torch.Generator().manual_seed(2)
        x[torch.rand(30, vocab, generator=g) < 0.4] = -INF
        x[torch.rand(30, vocab, generator=g) < 0.1] = float("nan")
        x[:, 1] = torch.finfo(dtype).min
        x[3], x[4] = -INF, float("nan")
        x[5], x[6] = torch.finfo(dtype).min, torch.finfo(dtype).min
        x[6, 2] = 0.0
        x[7] = -INF
        x[7, vocab - 1] = -3.0
        for s in SETTINGS:
            got = check(canon, x, u, **s)
            assert got[3] == -1 and got[4] == -1 and got[7] == vocab - 1
            # next to 0 the lowest value weighs nothing, but at an infinite temperature
            assert got[6] == 2 or s.get("temperature") == INF


def test_infinite_logits(canon):
    """The infinite ones share the whole weight."""
    x, u = logits(F32, 64, 50)
    x[:, 7] = x[:, 30] = x[:, 31] = INF
    u = torch.arange(64) / 64
    for s in (dict(), dict(top_p=0.9), dict(temperature=INF), dict(min_p=0.5), dict(top_k=10)):
        got = canon.sample(x.cuda(), u.cuda(), **s).cpu()
        want = torch.tensor([7, 30, 31])[(3 * u).long()]
        assert torch.equal(got, want), s
    assert (canon.sample(x.cuda(), u.cuda(), top_k=2).cpu() ==
            torch.tensor([7, 30])[(2 * u).long()]).all()
    assert (canon.sample(x.cuda(), u.cuda(), temperature=0.0) == 7).all()


def test_ties_go_to_the_lowest_index(canon):
    """Equal logits: weights are exactly 1, so every border is exact."""
    for vocab in (16, 2048, 33000):
        n = 64
        u = (torch.arange(n) / n).cuda()
        x = torch.zeros(n, vocab, device="cuda")
        x[:, ::2] = -0.0  # the same number
        assert torch.equal(canon.sample(x, u).cpu(), torch.arange(n) * vocab // n)
        # kept: the first tokens
        for s, kept in ((dict(top_k=8), 8), (dict(top_p=0.5), vocab // 2),
                        (dict(top_k=8, top_p=0.75), 6), (dict(top_p=0.0), 1)):
            got = canon.sample(x, u, **s).cpu()
            assert torch.equal(got, (torch.arange(n) * kept // n)), (vocab, s)
        # two levels: the higher ones first, then the lowest indexes among the others
        x[:, vocab // 2:vocab // 2 + 4] = 30.0
        got = canon.sample(x, u, temperature=1e6, top_k=8).cpu()
        order = torch.tensor([0, 1, 2, 3] + [vocab // 2 + i for i in range(4)])
        w = torch.tensor([math.exp(-30 / 1e6)] * 4 + [1.0] * 4, dtype=torch.float64)
        cum = torch.cumsum(w, 0) / w.sum()
        assert torch.equal(got, order[torch.searchsorted(cum, u.double().cpu(), right=True)])


def test_the_ends_of_u(canon):
    """0 takes the first kept token, 1 and beyond the last, NaN counts as 0."""
    x, _ = logits(F32, 6, 300, scale=1.0)
    x[:, 0] = x[:, 299] = -INF
    u = torch.tensor([0.0, -1.0, float("nan"), 1.0, 5.0, INF])
    assert canon.sample(x.cuda(), u.cuda()).tolist() == [1, 1, 1, 298, 298, 298]
    x[:, 200:] -= 100.0  # weights of zero: never taken
    assert canon.sample(x.cuda(), u.cuda()).tolist() == [1, 1, 1, 199, 199, 199]


def test_shares(canon):
    """Over a grid of u every token gets its share of the softmax."""
    x = torch.tensor([[0.5, -1.0, 2.0, 0.0, 1.0]])
    n = 1 << 16
    u = (torch.arange(n) + 0.5) / n
    got = canon.sample(x.expand(n, 5).cuda(), u.cuda(), temperature=0.8)
    share = torch.bincount(got.cpu(), minlength=5) / n
    assert (share - torch.softmax(x[0] / 0.8, 0)).abs().max() <= 2.0 / n


def test_layouts(canon):
    """Rows of a wider buffer at any start, int32 tokens, an output of the caller's."""
    for dtype in (F32, BF16):
        x, u = logits(dtype, 11, 2001, seed=3)
        want = canon.sample(x.cuda(), u.cuda(), top_p=0.9)
        big = torch.full((11, 2013), 50.0, dtype=dtype, device="cuda")
        big[:, 5:2006] = x.cuda()
        assert torch.equal(canon.sample(big[:, 5:2006], u.cuda(), top_p=0.9), want)
        out = torch.full((13,), 9, dtype=torch.int32, device="cuda")
        got = canon.sample(x.cuda(), u.cuda(), top_p=0.9, out=out[1:12])
        assert torch.equal(got.long(), want) and out[0] == 9 and out[12] == 9
        one = canon.sample(x[:1].cuda(), u[:1].cuda(), top_p=0.9)
        assert one[0] == want[0]


def test_nothing_to_do(canon):
    e = torch.empty(0, device="cuda")
    assert canon.sample(torch.empty(0, 9, device="cuda"), e).shape == (0,)
    assert canon.sample(torch.empty(2, 0, device="cuda"), torch.zeros(2, device="cuda")).tolist() \
        == [-1, -1]


def test_refusals(canon):
    x, u = (t.cuda() for t in logits(F32, 3, 20))
    for call, kind in (
            (lambda: canon.sample(x[0], u), ValueError),
            (lambda: canon.sample(x.double(), u), TypeError),
            (lambda: canon.sample(x.t(), torch.zeros(20, device="cuda")), ValueError),
            (lambda: canon.sample(x, u[:2]), ValueError),
            (lambda: canon.sample(x, u.double()), ValueError),
            (lambda: canon.sample(x, u, temperature=-1.0), ValueError),
            (lambda: canon.sample(x, u, temperature=float("nan")), ValueError),
            (lambda: canon.sample(x, u, top_k=-1), ValueError),
            (lambda: canon.sample(x, u, top_p=1.5), ValueError),
            (lambda: canon.sample(x, u, min_p=-0.1), ValueError),
            (lambda: canon.sample(x, u, top_k=torch.ones(3, device="cuda")), ValueError),
            (lambda: canon.sample(x, u, top_p=torch.ones(2, device="cuda")), ValueError),
            (lambda: canon.sample(x, u, temperature=torch.ones(3)), ValueError),
            (lambda: canon.sample(x, u, out=torch.empty(3, device="cuda")), TypeError),
            (lambda: canon.sample(x, u, out=torch.empty(2, dtype=torch.int64, device="cuda")),
             ValueError)):
        with pytest.raises(kind):
            call()
