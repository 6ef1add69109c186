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


def scan_grads(d, absolute=False):
    """selective_scan of everything (D, gate, softplus, states) and all gradients by
    the formulas, in float64, for sequences of one length side by side, on the
    tensors' device: d holds u, delta, z, dout [sequences, rows, channels], B, C
    [.., groups, states], A, D, bias, init, dfinal.  absolute: the sums of the
    absolute values of the terms instead."""
    e = {k: v.double() for k, v in d.items() if torch.is_tensor(v) and v.is_floating_point()}
    if absolute:
        for k in ("u", "B", "C", "D", "init", "dout", "dfinal"):
            e[k] = e[k].abs()
    raw = e["delta"] + e["bias"]
    dl = torch.nn.functional.softplus(raw, threshold=1e9)
    slope = torch.sigmoid(raw)
    A, size_A, z, q = e["A"], e["A"].abs() if absolute else e["A"], e["z"], torch.sigmoid(e["z"])
    gate, dgate = (z.abs(), 1.1 + z.abs()) if absolute else (z * q, q + z * q * (1 - q))
    groups = e["B"].shape[2]
    per = e["u"].shape[2] // groups

    def spread(x):
        return x.repeat_interleave(per, 1)

    rows, u = e["u"].shape[1], e["u"]
    h = [e["init"]]
    for t in range(rows):
        a = torch.exp(dl[:, t, :, None] * A)
        h.append(a * h[-1] + (dl[:, t] * u[:, t])[..., None] * spread(e["B"][:, t]))
    g = {k: torch.zeros_like(e[k]) for k in ("u", "delta", "A", "B", "C", "D", "z", "bias")}
    out = torch.zeros_like(u)
    R = e["dfinal"]
    for t in range(rows - 1, -1, -1):
        B, C = spread(e["B"][:, t]), spread(e["C"][:, t])
        y = (h[t + 1] * C).sum(-1) + e["D"] * u[:, t]
        out[:, t] = y * gate[:, t]
        dy = e["dout"][:, t] * gate[:, t]
        lam = C * dy[..., None] + R
        R = torch.exp(dl[:, t, :, None] * A) * lam
        decay, through = R * h[t], (lam * B).sum(-1)
        dd = ((decay * size_A).sum(-1) + through * u[:, t]) * slope[:, t]
        g["u"][:, t] = through * dl[:, t] + e["D"] * dy
        g["delta"][:, t] = dd
        g["z"][:, t] = e["dout"][:, t] * y * dgate[:, t]
        by_group = (y.shape[0], groups, per, -1)
        g["B"][:, t] = (lam * (dl[:, t] * u[:, t])[..., None]).view(by_group).sum(2)
        g["C"][:, t] = (h[t + 1] * dy[..., None]).view(by_group).sum(2)
        g["A"] += (decay * dl[:, t][..., None]).sum(0)
        g["D"] += (dy * u[:, t]).sum(0)
        g["bias"] += dd.sum(0)
    g["init"] = R
    return out, h[-1], g
