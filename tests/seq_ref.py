"""Plain float64 forms of the sequence operators, one sequence at a time, and
the error bounds the GPU tests use."""
import torch

U32 = 2.0 ** -24  # a float32 rounding, relative


def half_step(dtype):
    """Largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


def spans(x, starts):
    """(index into the leading dimensions of x) per sequence."""
    if starts is None:
        return [(s,) for s in range(x.shape[0])]
    p = starts.tolist()
    return [(slice(a, b),) for a, b in zip(p[:-1], p[1:])]


def silu(p):
    return p * torch.sigmoid(p)


def conv_one(x, w, b, act, init):
    """x [rows, channels], init [taps - 1, channels] -> out, final state"""
    k = w.shape[1]
    full = torch.cat([init, x])
    p = torch.zeros_like(x) if b is None else b + torch.zeros_like(x)
    for j in range(k):
        p = p + w[:, j] * full[j:j + x.shape[0]]
    return (silu(p) if act else p), full[x.shape[0]:]


def scan_one(u, delta, A, B, C, D, z, bias, softplus, h0):
    """u, delta, z [rows, channels]; B, C [rows, groups, states] -> out, final state"""
    raw = delta + (0 if bias is None else bias)
    dl = torch.nn.functional.softplus(raw, threshold=1e9) if softplus else raw
    per = u.shape[1] // B.shape[1]
    Bf, Cf = B.repeat_interleave(per, 1), C.repeat_interleave(per, 1)
    h, ys = h0, []
    for t in range(u.shape[0]):
        h = torch.exp(dl[t][:, None] * A) * h + (dl[t] * u[t])[:, None] * Bf[t]
        ys.append((h * Cf[t]).sum(-1))
    y = torch.stack(ys) if ys else torch.zeros_like(u)
    if D is not None:
        y = y + D * u
    return (y * silu(z) if z is not None else y), h


def close(got, want, size, terms, what=""):
    """|got - want| <= rounding of the stored value + terms float32 roundings of
    `size`, the sum of the absolute values of the terms that want adds up."""
    got64 = got.detach().double().cpu()
    want, size = want.detach(), size.detach()
    tol = terms * U32 * size + half_step(got.dtype) * (want.abs() + terms * U32 * size)
    tol = tol + float(torch.finfo(got.dtype).tiny)
    bad = ~((got64 - want).abs() <= tol)
    bad &= ~(torch.isnan(got64) & torch.isnan(want))
    assert not bad.any(), (
        f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound; worst "
        f"{float(((got64 - want).abs() / tol)[bad].max())} times it at "
        f"{torch.nonzero(bad)[0].tolist()}")
