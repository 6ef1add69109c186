"""Plain float64 forms of the layer operators and the error bounds the GPU tests
use: each a bound on the sum of the float32 roundings behind a value."""
import torch

U = 2.0 ** -24  # a float32 rounding, relative


def within(got, want, tol, what=""):
    """|got - want| <= tol + the rounding of the stored value, element by element."""
    want, tol = want.detach(), tol.detach()
    half = torch.finfo(got.dtype).eps / 2
    g = got.detach().double().cpu()
    limit = tol + half * (want.abs() + tol) + float(torch.finfo(got.dtype).tiny)
    bad = ~((g - want).abs() <= limit) & ~(torch.isnan(g) & torch.isnan(want))
    bad &= ~(torch.isinf(want) & (g == want))
    assert not bad.any(), (
        f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound; worst "
        f"{float(((g - want).abs() / limit)[bad].max())} times it at "
        f"{torch.nonzero(bad)[0].tolist()}")


# ------------------------------------------------------------------ layer norm
def norm_depth(width):
    """Additions one after the other in a sum over a row: a thread's vectors of at
    most 8 columns (a tree of 3 levels each, 256 threads or more wherever there is
    more than one vector), then at most 10 levels over the threads."""
    return width // 1024 + 16 + 13


def norm(x, w, b, eps):
    """float64: out, and a bound on its float32 evaluation; mean, rstd likewise."""
    x, w = x.double().cpu(), w.double().cpu()
    b = torch.zeros_like(w) if b is None else b.double().cpu()
    D = norm_depth(x.shape[-1])
    m = x.mean(-1, keepdim=True)
    d = x - m
    v = (d * d).mean(-1, keepdim=True)
    r = 1 / torch.sqrt(v + eps)
    # the sum's D roundings, the division's two
    em = (D + 3) * U * x.abs().mean(-1, keepdim=True)
    # squares of d (2 roundings each, and the mean's error, whose product with the
    # deviations adds up to zero and whose square stays), their sum, eps; halved by
    # the square root, whose own error is 2
    er = ((D + 8) / 2 + 2) * U + (em * r) ** 2
    out = d * r * w + b
    tol = w.abs() * r * (em + d.abs() * (er + 4 * U)) + 2 * U * (out.abs() + b.abs())
    return out, tol, (m, em), (r, r * er)


def norm_grad(dout, x, w, dsum, eps):
    """float64 gradients by the formula, with bounds: dx, dweight, dbias."""
    rows = x.reshape(-1, x.shape[-1]).shape[0]
    x, w, dout = x.double().cpu(), w.double().cpu(), dout.double().cpu()
    _, _, (m, em), (r, err) = norm(x, w, None, eps)
    D = norm_depth(x.shape[-1])
    er = err / r
    d = x - m
    n = d * r
    en = r * (em + U * d.abs()) + n.abs() * (er + 2 * U)
    g = dout * w
    s = g.mean(-1, keepdim=True)
    q = (g * n).mean(-1, keepdim=True)
    es = (D + 4) * U * g.abs().mean(-1, keepdim=True)
    eq = (D + 6) * U * (g * n).abs().mean(-1, keepdim=True) + (g.abs() * en).mean(-1, keepdim=True)
    core = g - s - n * q
    dx = r * core
    tol = (r * (4 * U * (g.abs() + s.abs() + (n * q).abs()) + es + n.abs() * eq + q.abs() * en)
           + (er + 2 * U) * dx.abs())
    if dsum is not None:
        dsum = dsum.double().cpu()
        dx = dx + dsum
        tol = tol + 2 * U * (dx.abs() + dsum.abs())
    # a chunk's rows (64 at most, 8 lanes), then the chunks by 16 lanes and a tree
    Dr = 64 + 4 + (max(512, rows // 64) // 16) + 5
    flat = tuple(range(x.dim() - 1))
    dw = (dout * n).sum(flat)
    tw = (Dr + 3) * U * (dout * n).abs().sum(flat) + (dout.abs() * en).sum(flat)
    return (dx, tol), (dw, tw), (dout.sum(flat), Dr * U * dout.abs().sum(flat))
