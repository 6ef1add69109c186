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


# ------------------------------------------------------ gated linear recurrence
BLOCK = 512  # rows


def recur_parts(gate, input_gate, decay):
    """float64: a, c, i, r, the slope -dc/d(log a), and whether a decay is given"""
    r = torch.sigmoid(gate)
    i = torch.ones_like(r) if input_gate is None else torch.sigmoid(input_gate)
    if decay is None:
        return r, torch.sigmoid(-gate), i, r, r
    log_a = -decay * r
    a = torch.exp(log_a)
    c = torch.sqrt(-torch.expm1(2 * log_a))
    return a, c, i, r, torch.where(c > 0, a * a / c.clamp(min=1e-300), torch.zeros_like(c))


def recur(x, gate, input_gate=None, decay=None, init=None, dout=None, dfinal=None):
    """Sequences of one length side by side, [sequences, rows, channels], in float64 on
    the CPU: a dict of (value, bound) for out, final and, with dout, x, gate, input_gate,
    decay, init.

    Bounds, in float32 roundings U.  The sigmoid of y has a relative error of (|y| + 4) U
    (its exponential's is |y| U and an ulp, the reciprocal's an ulp), e = a - 1 one of
    (|gate| + 16) U, c i x one of (|gate| + |input_gate| + 26) U.  A chunk folds 8 rows
    with two roundings each, relative to the absolute sum; the state at a round's start
    goes through a carry in 64 bits that takes the chunks' folds in 32 and is rounded 3
    times a block of 512 rows; an output adds the rounding of that state to 32 bits, two
    for each of at most 15 chunks of the round and the 16 of its own chunk, 47.  So with
    A the recurrence of absolute values, an error E obeys
      E <- a E + (48 + |gate|) U |e| A + (64 + |gate| + |input_gate|) U |c i x|.
    The decay's and its gate's gradients take a itself, as exp(l), l = log a, with a
    relative error of (|l| (|gate| + 5) + 1) U, or as 1 + e where |l| <= 1, with
    (|e| (|gate| + 16) + 1) U / a, at most (1.72 |l| (|gate| + 16) + 2.72) U: the latter
    bounds both, and counts twice for a^2.  An exp(l) below 2^-126, the least normal
    float32, is 0, off by less than 2^-126: a decay of 100 reaches l = -87.4, and its
    gradient that many times the least number."""
    f = {k: None if v is None else v.detach().double().cpu()
         for k, v in dict(x=x, g=gate, n=input_gate, D=decay, h=init, o=dout, F=dfinal).items()}
    x, g, n = f["x"], f["g"], f["n"]
    a, c, i, r, slope = recur_parts(g, n, f["D"])
    rows = x.shape[1]
    ng = torch.zeros_like(g) if n is None else n.abs()
    v = c * i * x
    ke = (48 + g.abs()) * U * (1 - a)
    kv = (64 + g.abs() + ng) * U
    zero = x.new_zeros(x.shape[0], x.shape[2])
    h, A = [f["h"] if f["h"] is not None else zero], [zero if f["h"] is None else f["h"].abs()]
    E, out, tol = zero, [], []
    T = [E + 3 * U * A[0]]
    for t in range(rows):
        E = a[:, t] * E + ke[:, t] * A[t] + kv[:, t] * v[:, t].abs()
        h.append(a[:, t] * h[t] + v[:, t])
        A.append(a[:, t] * A[t] + v[:, t].abs())
        if t % BLOCK == BLOCK - 1:
            E = E + 3 * U * A[-1]
        out.append(h[-1])
        tol.append(E + 48 * U * A[-1])
        T.append(E + 48 * U * A[-1])
    res = {"out": (torch.stack(out, 1), torch.stack(tol, 1)) if rows else (x, x),
           "final": (h[-1], E + 4 * U * A[-1])}
    if f["o"] is None:
        return res
    dout = f["o"]
    h, A, T = (torch.stack(q, 1) for q in (h, A, T))
    R = f["F"] if f["F"] is not None else zero  # what comes in past row t
    absR, E = R.abs(), zero
    lam, L, TL = (torch.zeros_like(x) for _ in range(3))
    for t in range(rows - 1, -1, -1):
        lam[:, t] = dout[:, t] + R
        L[:, t] = dout[:, t].abs() + absR
        TL[:, t] = E + 48 * U * L[:, t]
        E = a[:, t] * (E + 48 * U * dout[:, t].abs()) + ke[:, t] * L[:, t]
        R, absR = a[:, t] * lam[:, t], a[:, t] * L[:, t]
        if t % BLOCK == 0:
            E = E + 3 * U * absR
    res["init"] = (R, E + 4 * U * absR)
    res["x"] = (lam * c * i, c * i * (TL + L * kv))
    hp, Ap, Tp = h[:, :-1], A[:, :-1], T[:, :-1]
    ix = i * x
    if f["D"] is None:
        res["gate"] = (lam * (hp - ix) * a * c,
                       a * c * (TL * (Ap + ix.abs()) + L * (Tp + ix.abs() * U * (ng + 6))
                                + L * (Ap + ix.abs()) * U * (2 * g.abs() + 16)))
    else:
        B, absB = a * hp - slope * ix, a * Ap + slope * ix.abs()
        ka = 2 * U * (1.72 * f["D"] * r * (g.abs() + 16) + 2.72)
        bound = (TL * absB + L * (a * Tp + slope * ix.abs() * 2 * kv + (8 * U + ka) * absB
                                  + 2.0 ** -126 * Ap))
        dr = f["D"] * r * (1 - r)
        res["gate"] = (-dr * lam * B, dr * (bound + L * absB * U * (2 * g.abs() + 16)))
        blocks = x.shape[0] * (rows // BLOCK + 1)
        res["decay"] = (-(r * lam * B).sum((0, 1)),
                        (r * (bound + L * absB * U * (g.abs() + 8))).sum((0, 1))
                        + (64 + 10 + blocks // 16) * U * (r * L * absB).sum((0, 1)))
    if n is not None:
        res["input_gate"] = (lam * c * ix * (1 - i),
                             c * ix.abs() * (1 - i) * (TL + L * (kv + U * (ng + 10))))
    return res


# -------------------------------------------------------------------- sampling
def sample(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """The token of one row by a sort and sums in 80-bit numbers (64 bits of
    significand), and how far u is from the nearest token's border (1 where nothing
    depends on it), and top_p from the nearest sum, in shares of the whole."""
    import numpy as np
    x = np.where(np.isnan(x), -np.inf, x.astype(np.longdouble))
    order = np.lexsort((np.arange(x.size), -x))
    order = order[x[order] > -np.inf]
    if order.size == 0:
        return -1, 1.0
    if not temperature > 0:
        return int(order[0]), 1.0
    if top_k > 0:
        order = order[:top_k]
    top = x[order[0]]
    with np.errstate(invalid="ignore"):
        w = np.where(x[order] == top, np.longdouble(1),
                     np.exp((x[order] - top) / np.longdouble(temperature)))
    w = np.where(np.isnan(w), 0, w)
    margin = 1.0
    if top_p < 1:
        total = np.cumsum(w)
        want = np.longdouble(top_p) * total[-1]
        keep = 1 + int(np.searchsorted(total, want))
        margin = float(np.abs(total - want).min() / total[-1])
        order, w = order[:keep], w[:keep]
    keep = w >= min(min_p, 1.0)
    order, w = order[keep], w[keep]
    at = np.argsort(order)
    order, total = order[at], np.cumsum(w[at])
    want = np.longdouble(min(max(u, 0.0), 1.0)) * total[-1]
    margin = min(margin, float(np.abs(total[:-1] - want).min() / total[-1]) if total.size > 1
                 else 1.0)
    i = min(int(np.searchsorted(total, want, side="right")), order.size - 1)
    while w[at][i] == 0:  # u of 1
        i -= 1
    return int(order[i]), margin
