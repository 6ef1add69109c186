"""Cases of the sequence operators: embedding lookup and its gradient, the
short causal convolution, and the selective state space scan; prompts,
training passes and single tokens.

`run` computes a case in plain form (elementary torch operations in 32 bits)
or, where `own` is true, with the library's calls; `exact` computes it in 64
bits by another route.
"""
import math

import numpy as np
import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the tokens one decode step of a small server looks up: latency
        {"name": "embed_decode", "kind": "embed", "dtype": "f32", "tokens": 16, "rows": 50021,
         "width": 1024, "scale": 1.0, "pad": False},
        # the tokens of a padded batch of prompts, ids of padding outside the table
        {"name": "embed_prompts", "kind": "embed", "dtype": "bf16", "tokens": 16384,
         "rows": 65536, "width": 4096, "scale": 64.0, "pad": True},
        # gradient of a small batch, odd sizes, same type as the activations
        {"name": "embed_grad_odd", "kind": "embed_grad", "dtype": "f16", "grad": "f16",
         "tokens": 3001, "rows": 10007, "width": 1000, "scale": 1.0, "pad": True},
        # gradient of one training step: frequent and rare tokens, a 32-bit table
        {"name": "embed_grad_train", "kind": "embed_grad", "dtype": "bf16", "grad": "f32",
         "tokens": 16384, "rows": 65536, "width": 4096, "scale": 64.0, "pad": False},
        # packed prompts of different lengths continuing from cached inputs
        {"name": "conv_packed", "kind": "conv", "dtype": "bf16", "batch": 9, "length": 1777,
         "packed": True, "channels": 4096, "taps": 4, "silu": True, "state": True},
        # a training step's convolution, forward and backward
        {"name": "conv_train", "kind": "conv_train", "dtype": "bf16", "batch": 8, "length": 2048,
         "packed": False, "channels": 4096, "taps": 4, "silu": True, "state": False},
        # one token of each of a few sequences: latency
        {"name": "conv_step", "kind": "conv_step", "dtype": "bf16", "batch": 4,
         "channels": 2048, "taps": 4, "silu": True},
        # one long prompt: one sequence has to fill the chip
        {"name": "scan_long", "kind": "scan", "dtype": "bf16", "batch": 1, "length": 16384,
         "packed": False, "channels": 2048, "groups": 1, "states": 16, "gate": True,
         "state": True},
        # packed prompts, odd width, two groups of input and output maps
        {"name": "scan_packed_odd", "kind": "scan", "dtype": "f16", "batch": 7, "length": 701,
         "packed": True, "channels": 1000, "groups": 2, "states": 16, "gate": False,
         "state": True},
        # a training step's scan, forward and backward
        {"name": "scan_train", "kind": "scan_train", "dtype": "bf16", "batch": 8,
         "length": 2048, "packed": False, "channels": 4096, "groups": 1, "states": 16,
         "gate": True, "state": False},
        # a small 32-bit training step of odd sizes on packed sequences
        {"name": "scan_train_odd", "kind": "scan_train", "dtype": "f32", "batch": 3,
         "length": 333, "packed": True, "channels": 520, "groups": 1, "states": 8,
         "gate": False, "state": True},
        # one token of each sequence of a large serving batch
        {"name": "scan_step", "kind": "scan_step", "dtype": "bf16", "batch": 256,
         "channels": 4096, "groups": 1, "states": 16, "gate": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["embed", "embed_grad", "embed_grad", "conv", "conv_train", "conv_step",
                       "scan", "scan", "scan_train", "scan_train", "scan_step"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if kind in ("embed", "embed_grad"):
        case = {"kind": kind, "dtype": dtype, "tokens": _log(rng, 1, 8192),
                "rows": _log(rng, 100, 65536), "width": _log(rng, 64, 4096),
                "scale": rng.choice([1.0, 64.0]), "pad": rng.random() < 0.5}
        if kind == "embed_grad":
            case["grad"] = rng.choice([dtype, "f32"])
        return case
    channels = rng.choice([_log(rng, 64, 4096), 64 * _log(rng, 1, 64)])
    if kind == "conv_step":
        return {"kind": kind, "dtype": dtype, "batch": _log(rng, 1, 512), "channels": channels,
                "taps": rng.randint(2, 4), "silu": rng.random() < 0.8}
    groups = 2 if channels % 2 == 0 and rng.random() < 0.3 else 1
    states = rng.choice([4, 8, 13, 16, 16, 16])
    if kind == "scan_step":
        return {"kind": kind, "dtype": dtype, "batch": _log(rng, 1, 256), "channels": channels,
                "groups": groups, "states": states, "gate": rng.random() < 0.7}
    batch = _log(rng, 1, 16)
    length = _log(rng, 1, 16384 // batch)
    case = {"kind": kind, "dtype": dtype, "batch": batch, "length": length,
            "packed": rng.random() < 0.5, "channels": channels, "state": rng.random() < 0.5}
    if kind in ("conv", "conv_train"):
        if dtype == "f32":
            case["channels"] = min(channels, 2048)  # no more bytes than the listed cases
        case.update(taps=rng.randint(2, 4), silu=rng.random() < 0.8)
    else:
        if kind == "scan":  # no more work than the long prompt
            case["channels"] = min(channels, 1024 if dtype == "f32" else 2048)
        elif dtype == "f32":
            case["channels"] = min(channels, 2048)
        case["groups"] = groups if case["channels"] % 2 == 0 else 1
        case.update(states=states, gate=rng.random() < 0.7)
    return case


def _lengths(case):
    """Sequence lengths: equal, or for packed sequences from 0 to twice the
    mean, the same for every seed so that a case's work is its own."""
    n, mean = case["batch"], case["length"]
    if not case["packed"]:
        return [mean] * n
    total, lens = n * mean, []
    for i in range(n - 1):
        lens.append(min((2 * mean * ((i * 5 + 3) % n)) // n, total - sum(lens)))
    return lens + [total - sum(lens)]


def work(case):
    e = _SIZE[case["dtype"]]
    kind = case["kind"]
    if kind in ("embed", "embed_grad"):
        t, v, d = case["tokens"], case["rows"], case["width"]
        if kind == "embed":
            return {"bytes": 8 * t + (min(t, v) + t) * d * e, "flops": t * d}
        return {"bytes": 8 * t + t * d * e + v * d * _SIZE[case["grad"]], "flops": 2 * t * d}
    d = case["channels"]
    if kind == "conv_step":
        b, k = case["batch"], case["taps"]
        return {"bytes": b * d * e * (2 + 2 * (k - 1)) + d * 4 * (k + 1),
                "flops": b * d * (2 * k + 6)}
    if kind == "scan_step":
        b, n, g = case["batch"], case["states"], case["groups"]
        return {"bytes": b * d * (8 * n + e * (4 if case["gate"] else 3)) + 2 * b * g * n * e
                + 4 * d * (n + 2), "flops": b * d * (7 * n + 16)}
    b = case["batch"]
    t = b * case["length"]
    if kind in ("conv", "conv_train"):
        k = case["taps"]
        state = 2 * b * d * (k - 1) * e if case["state"] else 0
        if kind == "conv":
            return {"bytes": 2 * t * d * e + state + 4 * d * (k + 1), "flops": t * d * (2 * k + 6)}
        return {"bytes": 4 * t * d * e + state + 8 * d * (k + 1),
                "flops": t * d * (8 * k + 16)}
    n, g = case["states"], case["groups"]
    gate = 1 if case["gate"] else 0
    state = 8 * b * d * n if case["state"] else 0
    if kind == "scan":
        return {"bytes": t * d * e * (3 + gate) + 2 * t * g * n * e + state + 4 * d * (n + 2),
                "flops": t * d * (7 * n + 16)}
    return {"bytes": t * d * e * (6 + 2 * gate) + 4 * t * g * n * e + state + 8 * d * (n + 2),
            "flops": t * d * (23 * n + 40)}


# ------------------------------------------------------------------ the inputs
def _zipf(n, rows, gen):
    """Token ids with frequencies falling as 1/rank, ranks spread over the table."""
    r = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    rank = torch.exp(r * math.log(rows)).long().clamp_(1, rows) - 1
    step = 7919 if rows % 7919 else 7907
    return (rank * step + 17) % rows


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = _DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dt=dtype):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dt)

    kind = case["kind"]
    s = {"case": case}
    if kind in ("embed", "embed_grad"):
        t, v, d = case["tokens"], case["rows"], case["width"]
        ids = _zipf(t, v, gen)
        if case["pad"]:  # padding of a ragged batch
            ids[torch.rand(t, generator=gen, device="cuda") < 0.1] = -1
        s["ids"] = ids
        if kind == "embed":
            s["weight"] = normal(v, d, scale=0.02)
        else:
            s["dout"] = normal(t, d, scale=0.05)
        return s
    b, d = case["batch"], case["channels"]
    f32 = torch.float32
    if "taps" in case:
        k = case["taps"]
        s["weight"] = normal(d, k, scale=k ** -0.5, dt=f32)
        s["bias"] = normal(d, scale=0.1, dt=f32)
        s["activation"] = "silu" if case["silu"] else None
    else:
        n, g = case["states"], case["groups"]
        base = torch.arange(1, n + 1, device="cuda", dtype=f32)
        s["A"] = -(base * torch.exp(normal(d, n, scale=0.2, dt=f32)))
        s["D"] = 1.0 + normal(d, scale=0.2, dt=f32)
        # step sizes between 0.001 and 0.1 at a zero input
        dt0 = torch.exp(torch.rand(d, generator=gen, device="cuda") * math.log(100.0)) * 1e-3
        s["delta_bias"] = dt0 + torch.log(-torch.expm1(-dt0))
    if kind == "conv_step":
        s["x"] = normal(b, d)
        s["state"] = normal(b, case["taps"] - 1, d)
        return s
    if kind == "scan_step":
        s["u"], s["delta"] = normal(b, d), normal(b, d, scale=0.5)
        s["z"] = normal(b, d) if case["gate"] else None
        s["B"], s["C"] = normal(b, g, n), normal(b, g, n)
        s["state"] = normal(b, d, n, scale=0.3, dt=f32)
        return s
    lens = _lengths(case)
    lead = (sum(lens),) if case["packed"] else (b, case["length"])
    s["lens"] = lens
    s["starts"] = None
    if case["packed"]:
        s["starts"] = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
    train = kind.endswith("train")
    if "taps" in case:
        s["x"] = normal(*lead, d)
        s["init_state"] = normal(b, case["taps"] - 1, d) if case["state"] else None
        s["final_state"] = (torch.empty(b, case["taps"] - 1, d, dtype=dtype, device="cuda")
                            if case["state"] and not train else None)
    else:
        s["u"], s["delta"] = normal(*lead, d), normal(*lead, d, scale=0.5)
        s["z"] = normal(*lead, d) if case["gate"] else None
        s["B"], s["C"] = normal(*lead, g, n), normal(*lead, g, n)
        s["init_state"] = normal(b, d, n, scale=0.3, dt=f32) if case["state"] else None
        s["final_state"] = (torch.empty(b, d, n, dtype=f32, device="cuda")
                            if case["state"] and not train else None)
    if train:
        s["dout"] = normal(*lead, d)
    return s


# ------------------------------------------------------------- the library's calls
def _run_own(s):
    import scan_canonical_reduce_amd as canon

    case = s["case"]
    kind = case["kind"]
    if kind == "embed":
        return canon.embedding(s["weight"], s["ids"], scale=case["scale"])
    if kind == "embed_grad":
        return canon.embedding_grad(s["dout"], s["ids"], case["rows"], scale=case["scale"],
                                    dtype=_DTYPES[case["grad"]])
    if kind == "conv_step":
        nxt = torch.empty_like(s["state"])
        out = canon.causal_conv_step(s["x"], s["state"], s["weight"], s["bias"],
                                     activation=s["activation"], out_state=nxt)
        return out, nxt
    if kind == "scan_step":
        nxt = torch.empty_like(s["state"])
        out = canon.selective_scan_step(s["state"], s["u"], s["delta"], s["A"], s["B"], s["C"],
                                        D=s["D"], z=s["z"], delta_bias=s["delta_bias"],
                                        delta_softplus=True, out_state=nxt)
        return out, nxt
    if kind in ("conv", "conv_train"):
        out = canon.causal_conv(s["x"], s["weight"], s["bias"], activation=s["activation"],
                                starts=s["starts"], init_state=s["init_state"],
                                final_state=s["final_state"])
        if kind == "conv":
            return (out, s["final_state"]) if case["state"] else (out,)
        g = canon.causal_conv_grad(s["dout"], s["x"], s["weight"], s["bias"],
                                   activation=s["activation"], starts=s["starts"],
                                   init_state=s["init_state"])
        return (out, g.dx, g.dweight, g.dbias) + ((g.dinit_state,) if case["state"] else ())
    extra = dict(D=s["D"], z=s["z"], delta_bias=s["delta_bias"], delta_softplus=True,
                 starts=s["starts"])
    if kind == "scan":
        out = canon.selective_scan(s["u"], s["delta"], s["A"], s["B"], s["C"],
                                   init_state=s["init_state"], final_state=s["final_state"],
                                   **extra)
        return (out, s["final_state"]) if case["state"] else (out,)
    states = canon.selective_scan_states(s["u"], case["states"], s["starts"])
    out = canon.selective_scan(s["u"], s["delta"], s["A"], s["B"], s["C"],
                               init_state=s["init_state"], states=states, **extra)
    g = canon.selective_scan_grad(s["dout"], s["u"], s["delta"], s["A"], s["B"], s["C"], states,
                                  **extra)
    return ((out, g.du, g.ddelta, g.dA, g.dB, g.dC, g.dD, g.ddelta_bias)
            + ((g.dz,) if case["gate"] else ()) + ((g.dinit_state,) if case["state"] else ()))


# ---------------------------------------------------------------- the plain forms
def _pad(x, s):
    """[sequences, longest, ...] in 32 bits, packed sequences padded with 0."""
    if s["starts"] is None:
        return x.float()
    out = x.new_zeros((len(s["lens"]), max(s["lens"])) + x.shape[1:], dtype=torch.float32)
    at = 0
    for i, n in enumerate(s["lens"]):
        out[i, :n] = x[at:at + n]
        at += n
    return out


def _unpad(x, s, dtype):
    if s["starts"] is None:
        return x.to(dtype)
    return torch.cat([x[i, :n] for i, n in enumerate(s["lens"])]).to(dtype)


def _silu_grad(p):
    q = torch.sigmoid(p)
    return q * (1.0 + p * (1.0 - q))


def _conv_plain(s, backward):
    case = s["case"]
    dtype, k = s["x"].dtype, case["taps"]
    x, w = _pad(s["x"], s), s["weight"]
    n, length, d = x.shape
    head = s["init_state"].float() if s["init_state"] is not None else x.new_zeros(n, k - 1, d)
    full = torch.cat([head, x], 1)
    p = s["bias"] + full[:, :length] * w[:, 0]
    for j in range(1, k):
        p = p + full[:, j:j + length] * w[:, j]
    out = _unpad(p * torch.sigmoid(p) if case["silu"] else p, s, dtype)
    if not backward:
        if not case["state"]:
            return (out,)
        last = torch.stack([full[i, m:m + k - 1] for i, m in enumerate(s["lens"])])
        return out, last.to(dtype)
    dp = _pad(s["dout"], s)
    if case["silu"]:
        dp = dp * _silu_grad(p)
    dfull = torch.zeros_like(full)
    dw = []
    for j in range(k):
        dfull[:, j:j + length] += dp * w[:, j]
        dw.append((dp * full[:, j:j + length]).sum((0, 1)))
    res = (out, _unpad(dfull[:, k - 1:], s, dtype), torch.stack(dw, 1), dp.sum((0, 1)))
    return res + ((dfull[:, :k - 1].to(dtype),) if case["state"] else ())


def _spread(x, d):
    """B or C of each group for each of its channels."""
    return x if x.shape[-2] == 1 else x.repeat_interleave(d // x.shape[-2], -2)


def _scan_plain(s, backward):
    case = s["case"]
    dtype = s["u"].dtype
    u, A = _pad(s["u"], s), s["A"]
    raw = _pad(s["delta"], s) + s["delta_bias"]
    dl = torch.where(raw > 20, raw, torch.log1p(torch.exp(raw.clamp(max=20))))
    if s["starts"] is not None:  # padding leaves the state as it is
        ends = torch.tensor(s["lens"], device=u.device)[:, None]
        dl = dl * (torch.arange(u.shape[1], device=u.device) < ends)[..., None]
    B, C = _spread(_pad(s["B"], s), u.shape[2]), _spread(_pad(s["C"], s), u.shape[2])
    n, length, d = u.shape
    a = torch.exp(dl[..., None] * A).transpose(0, 1).contiguous()
    h = torch.empty(length + 1, n, d, case["states"], device=u.device)
    h[1:] = ((dl * u)[..., None] * B).transpose(0, 1)
    h[0] = s["init_state"] if s["init_state"] is not None else 0.0
    for t in range(length):
        h[t + 1].addcmul_(a[t], h[t])
    y = (h[1:].transpose(0, 1) * C).sum(-1) + s["D"] * u
    out = y
    if case["gate"]:
        z = _pad(s["z"], s)
        out = y * z * torch.sigmoid(z)
    out = _unpad(out, s, dtype)
    if not backward:
        return (out, h[length].clone()) if case["state"] else (out,)
    dout = _pad(s["dout"], s)
    dy = dout * z * torch.sigmoid(z) if case["gate"] else dout
    lam = (dy[..., None] * C).transpose(0, 1).contiguous()
    for t in range(length - 1, 0, -1):
        lam[t - 1].addcmul_(a[t], lam[t])
    dinit = a[0] * lam[0]
    dC = dy[..., None] * h[1:].transpose(0, 1)
    decay = (lam * a * h[:length]).transpose(0, 1)
    lam = lam.transpose(0, 1)
    dB = (dl * u)[..., None] * lam
    g = case["groups"]
    dB = dB.view(n, length, g, d // g, -1).sum(3)
    dC = dC.view(n, length, g, d // g, -1).sum(3)
    through = (lam * B).sum(-1)
    ddl = (decay * A).sum(-1) + through * u
    dA = (decay * dl[..., None]).sum((0, 1))
    draw_ = ddl * torch.where(raw > 20, torch.ones_like(raw), torch.sigmoid(raw))
    if s["starts"] is not None:
        draw_ = draw_ * (dl != 0)
    du = through * dl + s["D"] * dy
    res = (out, _unpad(du, s, dtype), _unpad(draw_, s, dtype), dA, _unpad(dB, s, dtype),
           _unpad(dC, s, dtype), (dy * u).sum((0, 1)), draw_.sum((0, 1)))
    if case["gate"]:
        res += (_unpad(dout * y * _silu_grad(z), s, dtype),)
    return res + ((dinit,) if case["state"] else ())


def run(s):
    if own:
        return _run_own(s)
    case = s["case"]
    kind = case["kind"]
    if kind == "embed":
        w, ids = s["weight"], s["ids"]
        ok = (ids >= 0) & (ids < case["rows"])
        y = w[torch.where(ok, ids, 0)].float() * case["scale"] * ok[:, None]
        return y.to(w.dtype)
    if kind == "embed_grad":
        ids = s["ids"]
        ok = (ids >= 0) & (ids < case["rows"])
        dw = torch.zeros(case["rows"], case["width"], device=ids.device)
        dw.index_add_(0, torch.where(ok, ids, 0), s["dout"].float() * ok[:, None])
        return (dw * case["scale"]).to(_DTYPES[case["grad"]])
    if kind == "conv_step":
        x, w = s["x"].float(), s["weight"]
        full = torch.cat([s["state"].float(), x[:, None]], 1)
        p = s["bias"] + (full * w.t()).sum(1)
        y = p * torch.sigmoid(p) if case["silu"] else p
        return y.to(s["x"].dtype), full[:, 1:].to(s["x"].dtype)
    if kind == "scan_step":
        u, d = s["u"].float(), case["channels"]
        raw = s["delta"].float() + s["delta_bias"]
        dl = torch.where(raw > 20, raw, torch.log1p(torch.exp(raw.clamp(max=20))))
        B, C = _spread(s["B"].float(), d), _spread(s["C"].float(), d)
        h = torch.exp(dl[..., None] * s["A"]) * s["state"] + (dl * u)[..., None] * B
        y = (h * C).sum(-1) + s["D"] * u
        if case["gate"]:
            z = s["z"].float()
            y = y * z * torch.sigmoid(z)
        return y.to(s["u"].dtype), h
    if kind in ("conv", "conv_train"):
        return _conv_plain(s, kind == "conv_train")
    return _scan_plain(s, kind == "scan_train")


# ------------------------------------------------------------------------- exact
def _fold64(a, b, h0):
    """h[t] = a[t] h[t-1] + b[t] along dimension 0, by doubling; destroys a and b."""
    b[0] += a[0] * h0
    n, step = a.shape[0], 1
    while step < n:
        b[step:] += a[step:] * b[:-step].clone()
        a[step:] *= a[:-step].clone()
        step *= 2
    return b


def _exact_conv(s, backward):
    case = s["case"]
    k, d = case["taps"], case["channels"]
    w, bias = s["weight"].double(), s["bias"].double()
    x = s["x"].double().reshape(-1, d)
    outs, finals, dxs, dinits = [], [], [], []
    dw, db = torch.zeros_like(w), torch.zeros_like(bias)
    at = 0
    for i, n in enumerate(s["lens"]):
        head = (s["init_state"][i].double() if s["init_state"] is not None
                else x.new_zeros(k - 1, d))
        full = torch.cat([head, x[at:at + n]])
        win = full.unfold(0, k, 1) if n else x.new_zeros(0, d, k)  # [n, d, k]
        p = (win * w).sum(-1) + bias
        q = 1.0 / (1.0 + torch.exp(-p))
        outs.append(p * q if case["silu"] else p)
        finals.append(full[n:])
        if backward:
            g = s["dout"].reshape(-1, d)[at:at + n].double()
            if case["silu"]:
                g = g * (q + p * q * (1.0 - q))
            dw += (win * g[..., None]).sum(0)
            db += g.sum(0)
            # dfull[m] = sum_j w[j] g[m - j]
            pad = torch.cat([g.new_zeros(k - 1, d), g, g.new_zeros(k - 1, d)])
            dfull = (pad.unfold(0, k, 1) * w.flip(1)).sum(-1)
            dinits.append(dfull[:k - 1])
            dxs.append(dfull[k - 1:])
        at += n
    shape = s["x"].shape
    out = torch.cat(outs).view(shape)
    if not backward:
        return (out, torch.stack(finals)) if case["state"] else (out,)
    res = (out, torch.cat(dxs).view(shape), dw, db)
    return res + ((torch.stack(dinits),) if case["state"] else ())


def _exact_scan(s, backward):
    case = s["case"]
    d, n, g = case["channels"], case["states"], case["groups"]
    shape = s["u"].shape
    flat = {k: s[k].reshape(-1, d) for k in ("u", "delta")}
    flat["z"] = s["z"].reshape(-1, d) if case["gate"] else None
    if backward:
        flat["dout"] = s["dout"].reshape(-1, d)
    B, C = s["B"].reshape(-1, g, n).double(), s["C"].reshape(-1, g, n).double()
    total = flat["u"].shape[0]
    dev = s["u"].device

    def new(*size):
        return torch.zeros(*size, dtype=torch.float64, device=dev)

    out, final = new(total, d), new(case["batch"], d, n)
    if backward:
        du, ddelta, dz = new(total, d), new(total, d), new(total, d)
        dA, dB, dC = new(d, n), new(total, g, n), new(total, g, n)
        dD, dbias, dinit = new(d), new(d), new(case["batch"], d, n)
    at = 0
    for i, length in enumerate(s["lens"]):
        rows = slice(at, at + length)
        at += length
        width = max(8, min(d // g, (1 << 26) // max(1, length * n)))
        for grp in range(g):
            for lo in range(grp * (d // g), (grp + 1) * (d // g), width):
                ch = slice(lo, min(lo + width, (grp + 1) * (d // g)))
                A = s["A"][ch].double()
                h0 = (s["init_state"][i, ch].double() if s["init_state"] is not None
                      else torch.zeros_like(A))
                if length == 0:
                    final[i, ch] = h0
                    if backward:
                        dinit[i, ch] = 0.0
                    continue
                u = flat["u"][rows, ch].double()
                raw = flat["delta"][rows, ch].double() + s["delta_bias"][ch].double()
                dl = torch.logaddexp(raw, torch.zeros_like(raw))
                b, c = B[rows, grp][:, None], C[rows, grp][:, None]
                a = torch.exp(dl[..., None] * A)
                h = _fold64(a.clone(), (dl * u)[..., None] * b, h0)
                Dc = s["D"][ch].double()
                y = (h * c).sum(-1) + Dc * u
                final[i, ch] = h[-1]
                gate = torch.ones_like(y)
                if case["gate"]:
                    z = flat["z"][rows, ch].double()
                    q = 1.0 / (1.0 + torch.exp(-z))
                    gate = z * q
                out[rows, ch] = y * gate
                if not backward:
                    continue
                go = flat["dout"][rows, ch].double()
                if case["gate"]:
                    dz[rows, ch] = go * y * (q + z * q * (1.0 - q))
                dy = go * gate
                # lam[t] = C dy + a[t+1] lam[t+1], folded from the end
                later = torch.cat([torch.zeros_like(a[:1]), a[1:].flip(0)])
                lam = _fold64(later, (dy[..., None] * c).flip(0), torch.zeros_like(h0)).flip(0)
                dinit[i, ch] = a[0] * lam[0]
                prev = torch.cat([h0[None], h[:-1]])
                decay = lam * a * prev
                dA[ch] += (decay * dl[..., None]).sum(0)
                dB[rows, grp] += (lam * (dl * u)[..., None]).sum(1)
                dC[rows, grp] += (h * dy[..., None]).sum(1)
                through = (lam * b).sum(-1)
                slope = 1.0 / (1.0 + torch.exp(-raw))
                dd = ((decay * A).sum(-1) + through * u) * slope
                ddelta[rows, ch] = dd
                dbias[ch] += dd.sum(0)
                du[rows, ch] = through * dl + Dc * dy
                dD[ch] += (dy * u).sum(0)
    out = out.view(shape)
    if not backward:
        return (out, final) if case["state"] else (out,)
    res = (out, du.view(shape), ddelta.view(shape), dA, dB.view(s["B"].shape),
           dC.view(s["C"].shape), dD, dbias)
    return (res + ((dz.view(shape),) if case["gate"] else ())
            + ((dinit,) if case["state"] else ()))


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "embed":
        y = torch.zeros(case["tokens"], case["width"], dtype=torch.float64, device="cuda")
        at = torch.nonzero((s["ids"] >= 0) & (s["ids"] < case["rows"]))[:, 0]
        y[at] = s["weight"].index_select(0, s["ids"][at]).double() * case["scale"]
        return y
    if kind == "embed_grad":
        dw = torch.zeros(case["rows"], case["width"], dtype=torch.float64, device="cuda")
        ids, order = torch.sort(s["ids"], stable=True)
        order = order[(ids >= 0) & (ids < case["rows"])]
        if order.numel():
            rows, counts = torch.unique_consecutive(s["ids"][order], return_counts=True)
            total = torch.cumsum(s["dout"][order].double(), 0)[torch.cumsum(counts, 0) - 1]
            dw[rows] = torch.diff(total, dim=0, prepend=torch.zeros_like(total[:1]))
        return dw * case["scale"]
    if kind == "conv_step":
        w = s["weight"].double()
        full = torch.cat([s["state"], s["x"][:, None]], 1).double()
        p = s["bias"].double() + sum(full[:, j] * w[:, j] for j in range(case["taps"]))
        return (p / (1.0 + torch.exp(-p)) if case["silu"] else p), full[:, 1:]
    if kind == "scan_step":
        d, g = case["channels"], case["groups"]
        u = s["u"].double()
        raw = s["delta"].double() + s["delta_bias"].double()
        dl = torch.logaddexp(raw, torch.zeros_like(raw))
        grp = torch.arange(d, device=u.device) // (d // g)
        h = (torch.exp(dl[..., None] * s["A"].double()) * s["state"].double()
             + (dl * u)[..., None] * s["B"].double()[:, grp])
        y = (h * s["C"].double()[:, grp]).sum(-1) + s["D"].double() * u
        if case["gate"]:
            z = s["z"].double()
            y = y * z / (1.0 + torch.exp(-z))
        return y, h
    if kind in ("conv", "conv_train"):
        return _exact_conv(s, kind == "conv_train")
    return _exact_scan(s, kind == "scan_train")
