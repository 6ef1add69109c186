"""Sampling at settings and logits where its steps of the logit reach their limits, against
a sort in 80-bit numbers."""
import math

import numpy as np
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


def margin(x, temperature=1.0):
    """What the kernel's rounding can shift a border of row x by, as a share of the sum of
    what is kept.  A weight is off by 2^-51 of itself and by half a step of 2^-S, S = 62 -
    ceil(log2 vocab), 50 at most; other roundings (of u or top_p times the sum in 64 bits) add
    2^-52.  What filters keep are the largest weights, whose mean is at least that of all: so
    the half steps are at most 2^-(S + 1) over the mean weight of all."""
    steps = min(50, 62 - max(0, math.ceil(math.log2(max(x.size, 1)))))
    x = x[x > -INF].astype("float64")
    return 2.0 ** -50 + 2.0 ** -(steps + 1) / np.exp((x - x.max()) / temperature).mean()


def check(canon, x, u, least=0.9, **settings):
    """Every row that lies further from a border than the rounding reaches: at least this
    share of them, and one."""
    on = {k: v.cuda() if torch.is_tensor(v) else v for k, v in settings.items()}
    got = canon.sample(x.cuda(), u.cuda(), **on).cpu()
    values, compared = x.float().numpy(), 0
    for i in range(len(x)):
        s = {k: v[i].item() if torch.is_tensor(v) else v for k, v in settings.items()}
        want, gap = layer_ref.sample(values[i], float(u[i]), **s)
        if gap > margin(values[i], s.get("temperature", 1.0)):
            compared += 1
            assert got[i] == want, (settings, i, int(got[i]), want)
    assert compared >= max(1, least * len(x)), (settings, compared, len(x))
    return got


def logits(dtype, rows, vocab, seed=0, scale=3.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, vocab, generator=g) * scale).to(dtype), torch.rand(rows, generator=g)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("vocab", [2, 9, 130, 700, 5000])
def test_high_temperatures(canon, dtype, vocab):
    """Above 14.2 the steps go by the row's range, whose least logit the waves exchange
    right after its largest, and most waves of a small vocabulary have no logit: thousands
    of rows, each as its own kind gives."""
    kinds, copies = 16, 256
    x, u = logits(dtype, kinds, vocab, seed=vocab)
    g = torch.Generator().manual_seed(1)
    for s in (dict(temperature=20.0, top_k=5), dict(temperature=1e4, top_k=max(2, vocab // 2)),
              dict(temperature=100.0, top_p=0.7), dict(temperature=INF, top_k=3, top_p=0.9),
              dict(temperature=INF, top_p=0.4137)):
        one = check(canon, x, u, least=0.5, **s)
        order = torch.randperm(kinds * copies, generator=g) % kinds
        many = canon.sample(x[order].cuda(), u[order].cuda(), **s).cpu()
        assert torch.equal(many, one[order]), s


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("vocab", [5, 300, 9000])
def test_logits_further_apart_than_the_largest_number(canon, dtype, vocab):
    """Temperatures at which a logit of -3e38 weighs something beside one of 3e38: the
    difference is beyond 32 bits, and filters count the low ones as any others."""
    u = torch.arange(40) / 40 + 1 / 80
    x = torch.full((40, vocab), -3e38)
    x[:, 2] = 3e38
    x = x.to(dtype)
    for t in (INF, 2e38):
        got = check(canon, x, u, temperature=t, top_k=2)
        assert set(got.tolist()) == {0, 2}
        check(canon, x, u, temperature=t, top_k=4)
        check(canon, x, u, temperature=t, top_k=4, top_p=0.7)
        check(canon, x, u, temperature=t, top_p=0.4137)
        check(canon, x, u, temperature=t)
    many = logits(dtype, 40, vocab, seed=vocab, scale=1e38)[0].clamp(-3.3e38, 3.3e38)
    for s in (dict(top_k=3), dict(top_k=3, top_p=0.8), dict(top_p=0.6137)):
        check(canon, many, u, least=0.5, temperature=1e38, **s)
        check(canon, many, u, least=0.5, temperature=1e30, **s)


def test_top_k_of_other_kinds(canon):
    """Integers of any kind and size; nothing else."""
    x, u = (t.cuda() for t in logits(F32, 3, 20))
    want = canon.sample(x, u, top_k=4)
    assert torch.equal(canon.sample(x, u, top_k=np.int64(4)), want)
    everything = canon.sample(x, u)
    for k in (20, 21, 1 << 31, (1 << 32) + 1, 1 << 70):
        assert torch.equal(canon.sample(x, u, top_k=k), everything)
    for k in (4.0, "4", None):
        with pytest.raises(TypeError):
            canon.sample(x, u, top_k=k)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("vocab", [131072, 700001, (1 << 20) + 3])
def test_large_vocabularies(canon, dtype, vocab):
    """Four rows in five and more further from every border than the weights' rounding."""
    x, u = logits(dtype, 5, vocab, seed=vocab)
    for s in (dict(), dict(top_p=0.9), dict(top_k=50), dict(top_k=3000, top_p=0.8),
              dict(temperature=0.7, min_p=0.01), dict(temperature=30.0, top_k=40000)):
        check(canon, x, u, least=0.8, **s)
