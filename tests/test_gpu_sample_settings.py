"""Sampling at settings and logits where its steps of the logit reach their limits, against
a sort in 80-bit numbers."""
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


def margin(vocab):
    """What the kernel's rounding can shift a border by, as a share of the whole, which is
    one at least: a weight is off by 2^-51 of itself and by half a step of 2^-S, S = 62 -
    ceil(log2 vocab), 50 at most; a sum's other roundings (u or top_p times it in 64 bits)
    add 2^-52.  2^-28 at 2^17 tokens, 2^-36 at 2^13."""
    steps = min(50, 62 - max(0, math.ceil(math.log2(max(vocab, 1)))))
    return 2.0 ** -50 + vocab * 2.0 ** -(steps + 1)


def check(canon, x, u, least=0.9, **settings):
    """Every row that lies further from a border than the rounding reaches: at least this
    share of them, and one."""
    on = {k: v.cuda() if torch.is_tensor(v) else v for k, v in settings.items()}
    got = canon.sample(x.cuda(), u.cuda(), **on).cpu()
    values, compared = x.float().numpy(), 0
    for i in range(len(x)):
        s = {k: v[i].item() if torch.is_tensor(v) else v for k, v in settings.items()}
        want, gap = layer_ref.sample(values[i], float(u[i]), **s)
        if gap > margin(x.shape[1]):
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
