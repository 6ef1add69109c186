"""Layer norm against its float64 form: forward, residual sum, backward."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import layer_ref  # noqa: E402

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
EPS = 1e-5


@pytest.fixture(scope="module")
def canon():
    import scan_canonical_reduce_amd as c
    return c


def inputs(dtype, rows, width, param=F32, seed=0, mean=0.0):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g)

    shape = rows if isinstance(rows, tuple) else (rows,)
    return {k: v.cuda() for k, v in dict(
        x=(normal(*shape, width) + mean).to(dtype), res=(2 * normal(*shape, width)).to(dtype),
        w=(1 + 0.3 * normal(width)).to(param), b=(0.2 * normal(width)).to(param),
        dout=normal(*shape, width).to(dtype), dsum=normal(*shape, width).to(dtype)).items()}


WIDTHS = [1, 2, 7, 8, 31, 64, 65, 128, 200, 256, 257, 1000, 1021, 1024, 1025, 2048, 4095, 4096,
          4104, 8192, 16384, 16390, 20000, 32768, 33003]


def check_forward(canon, d, param_bias=True):
    b = d["b"] if param_bias else None
    stats = canon.layer_norm_stats(d["x"])
    got = canon.layer_norm(d["x"], d["w"], b, EPS, stats=stats)
    out, tol, (m, em), (r, er) = layer_ref.norm(d["x"], d["w"], b, EPS)
    layer_ref.within(got, out, tol, "out")
    layer_ref.within(stats[..., :1], m, em, "mean")
    layer_ref.within(stats[..., 1:], r, er, "1 / standard deviation")
    again, total = canon.add_layer_norm(d["x"], d["res"], d["w"], b, EPS)
    want = (d["x"].float() + d["res"].float()).to(d["x"].dtype)
    assert torch.equal(total, want)
    assert torch.equal(again, canon.layer_norm(want, d["w"], b, EPS))
    return got, stats


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("width", WIDTHS)
def test_forward(canon, dtype, width):
    for rows in (1, 5, 37):
        check_forward(canon, inputs(dtype, rows, width, seed=rows))
    check_forward(canon, inputs(dtype, 3, width, param=dtype, seed=9), False)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_many_rows(canon, dtype):
    """More rows than workgroups at once."""
    for rows, width in ((20011, 24), (9001, 136), (5003, 520), (4001, 2056)):
        check_forward(canon, inputs(dtype, rows, width, seed=1))


def test_a_mean_far_from_zero(canon):
    for width in (100, 1000, 5000, 40000):
        check_forward(canon, inputs(F32, 4, width, mean=300.0))


def check_backward(canon, d, bias=True, dsum=True):
    stats = canon.layer_norm_stats(d["x"])
    canon.layer_norm(d["x"], d["w"], None, EPS, stats=stats)
    got = canon.layer_norm_grad(d["dout"], d["x"], d["w"], stats, bias=d["b"] if bias else None,
                                dsum=d["dsum"] if dsum else None)
    dx, dw, db = layer_ref.norm_grad(d["dout"], d["x"], d["w"], d["dsum"] if dsum else None, EPS)
    layer_ref.within(got.dx, *dx, "dx")
    layer_ref.within(got.dweight, *dw, "dweight")
    assert (got.dbias is None) != bias
    if bias:
        layer_ref.within(got.dbias, *db, "dbias")
    return got


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("width", WIDTHS)
def test_backward(canon, dtype, width):
    for rows in (1, 5, 37):
        check_backward(canon, inputs(dtype, rows, width, seed=rows), rows != 5, rows != 37)
    check_backward(canon, inputs(dtype, 3, width, param=dtype, seed=9))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows", [511, 512, 513, 1024, 1025, 40000])
def test_chunks_of_rows(canon, dtype, rows):
    check_backward(canon, inputs(dtype, rows, 72 if rows > 2000 else 264, seed=3))


def test_gradient_against_differences(canon):
    """The directional derivative of the float64 form by central differences (h of
    1e-5: an error below 1e-8 of the loss's third derivative, far below the bounds)
    against the kernel's gradients."""
    d = inputs(F32, 6, 50, seed=5)
    got = check_backward(canon, d, dsum=False)
    e = {k: v.double().cpu() for k, v in d.items()}
    g = torch.Generator().manual_seed(6)
    h = 1e-5
    for name, grad, tol in zip(
            ("x", "w", "b"), got,
            (t for _, t in layer_ref.norm_grad(d["dout"], d["x"], d["w"], None, EPS))):
        v = torch.randn(e[name].shape, generator=g, dtype=torch.float64)

        def loss(step):
            p = dict(e, **{name: e[name] + step * v})
            m = p["x"].mean(-1, keepdim=True)
            var = ((p["x"] - m) ** 2).mean(-1, keepdim=True)
            return float(((p["x"] - m) / torch.sqrt(var + EPS) * p["w"] + p["b"])
                         .mul(e["dout"]).sum())

        want = (loss(h) - loss(-h)) / (2 * h)
        limit = float(((tol + layer_ref.U * grad.double().cpu().abs()) * v.abs()).sum()) + 1e-7
        assert abs(float((grad.double().cpu() * v).sum()) - want) <= limit, name


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("width", [33, 250, 1000, 4098, 20001])
def test_a_row_alone(canon, dtype, width):
    """A row's bits depend on nothing but the row: alone, at any alignment, strided,
    in sequences, any number of rows."""
    d = inputs(dtype, 41, width, seed=7)
    out, total = canon.add_layer_norm(d["x"], d["res"], d["w"], d["b"], EPS)
    one, t1 = canon.add_layer_norm(d["x"][17:18], d["res"][17:18], d["w"], d["b"], EPS)
    assert torch.equal(one, out[17:18]) and torch.equal(t1, total[17:18])
    big = torch.zeros(41, width + 5, dtype=dtype, device="cuda")
    view = big[:, 3:width + 3]
    view.copy_(d["x"])
    dest = torch.full_like(big, 7.0)
    got, _ = canon.add_layer_norm(view, d["res"], d["w"], d["b"], EPS,
                                  out=dest[:, 1:width + 1])
    assert torch.equal(got, out)
    assert (dest[:, 0] == 7).all() and (dest[:, width + 1:] == 7).all()
    x3 = d["x"][:40].view(5, 8, width).transpose(0, 1)  # sequences of rows 5 apart
    got = canon.layer_norm(x3, d["w"], d["b"], EPS)
    assert torch.equal(got, canon.layer_norm(d["x"], d["w"], d["b"], EPS)[:40]
                       .view(5, 8, width).transpose(0, 1))


@pytest.mark.parametrize("width", [60, 1000, 4096, 40000])
def test_in_place(canon, width):
    d = inputs(BF16, 19, width, seed=8)
    out, total = canon.add_layer_norm(d["x"], d["res"], d["w"], d["b"], EPS)
    for a, b in (("x", "res"), ("res", "x")):
        x, r = d["x"].clone(), d["res"].clone()
        bufs = dict(x=x, res=r)
        got, t = canon.add_layer_norm(x, r, d["w"], d["b"], EPS, sum_out=bufs[a], out=bufs[b])
        assert torch.equal(got, out) and torch.equal(t, total)
    x = d["x"].clone()
    assert torch.equal(canon.layer_norm(x, d["w"], d["b"], EPS, out=x),
                       canon.layer_norm(d["x"], d["w"], d["b"], EPS))
    stats = canon.layer_norm_stats(total)
    canon.layer_norm(total, d["w"], None, EPS, stats=stats)
    want = canon.layer_norm_grad(d["dout"], total, d["w"], stats, d["b"], d["dsum"])
    for name in ("dout", "dsum"):
        c = {k: d[k].clone() for k in ("dout", "dsum")}
        got = canon.layer_norm_grad(c["dout"], total, d["w"], stats, d["b"], c["dsum"],
                                    dx=c[name])
        assert all(torch.equal(p, q) for p, q in zip(got, want)), name


def test_broadcast_rows(canon):
    """One residual row for all (stride 0)."""
    d = inputs(F32, 12, 100)
    r = d["res"][:1].expand(12, 100)
    assert torch.equal(canon.add_layer_norm(d["x"], r, d["w"], d["b"])[0],
                       canon.add_layer_norm(d["x"], r.contiguous(), d["w"], d["b"])[0])


def test_special_rows(canon):
    """A constant row normalises to its bias; rows that are not finite give NaN and
    leave the others alone."""
    for width in (40, 1500, 40000):
        d = inputs(F32, 6, width)
        want = canon.layer_norm(d["x"], d["w"], d["b"])
        x = d["x"].clone()
        x[1] = 0.25
        x[2, 3] = float("inf")
        x[4, width - 1] = float("nan")
        got = canon.layer_norm(x, d["w"], d["b"])
        assert torch.equal(got[1], d["b"])
        assert torch.isnan(got[2]).all() and torch.isnan(got[4]).all()
        for i in (0, 3, 5):
            assert torch.equal(got[i], want[i])


def test_nothing_to_do(canon):
    w = torch.ones(8, device="cuda")
    x = torch.empty(0, 8, device="cuda")
    assert canon.layer_norm(x, w).shape == (0, 8)
    g = canon.layer_norm_grad(x, x, w, canon.layer_norm_stats(x), bias=w)
    assert not g.dweight.any() and not g.dbias.any() and g.dx.shape == (0, 8)
    x = torch.empty(3, 0, device="cuda")
    e = torch.empty(0, device="cuda")
    assert canon.layer_norm(x, e).shape == (3, 0)
    assert canon.layer_norm_grad(x, x, e, canon.layer_norm_stats(x)).dweight.shape == (0,)


def test_refusals(canon):
    d = inputs(F32, 5, 16)
    x, w = d["x"], d["w"]
    stats = canon.layer_norm_stats(x)
    for call, kind in (
            (lambda: canon.layer_norm(x[0], w), ValueError),
            (lambda: canon.layer_norm(x.double(), w), TypeError),
            (lambda: canon.layer_norm(x, w.half()), TypeError),
            (lambda: canon.layer_norm(x, w[:8]), ValueError),
            (lambda: canon.layer_norm(x, w, d["b"].half()), ValueError),
            (lambda: canon.layer_norm(x.t(), w[:4]), ValueError),
            (lambda: canon.layer_norm(x, w, stats=stats[:2]), ValueError),
            (lambda: canon.layer_norm(x, w, out=x.half()), ValueError),
            (lambda: canon.layer_norm(x[1:4], w, out=x[1:].as_strided((3, 16), (17, 1))),
             ValueError),
            (lambda: canon.add_layer_norm(x, x[:2], w), ValueError),
            (lambda: canon.add_layer_norm(x, x, w, sum_out=stats), ValueError),
            (lambda: canon.add_layer_norm(x, d["res"], w, sum_out=x, out=x), ValueError),
            (lambda: canon.layer_norm_grad(x[:2], x, w, stats), ValueError),
            (lambda: canon.layer_norm_grad(d["dout"], x, w, stats, dx=x), ValueError),
            (lambda: canon.layer_norm(x, w.cpu()), ValueError)):
        with pytest.raises(kind):
            call()
