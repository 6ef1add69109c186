"""Cases of the layer operators beside the sequence operators: layer norm with its
residual sum, the gated linear recurrence, and sampling the next token; prompts,
training passes and single tokens.

`run` computes a case in plain form (elementary torch operations in 32 bits; in 64
the sampling's weights and sums and the recurrence, whose roundings add up over a
long memory) or, where `own` is true, with the library's calls; `exact` computes it in 64 bits or more by another route.
"""
import math

import numpy as np
import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2}
_EPS = 1e-5


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the rows one decode step of a small server normalises after a block: latency
        {"name": "norm_decode", "kind": "norm", "dtype": "bf16", "rows": 16, "width": 2048,
         "residual": True, "bias": True, "param": "f32"},
        # a training step's norm with the residual sum, forward and backward
        {"name": "norm_train", "kind": "norm_train", "dtype": "bf16", "rows": 16384,
         "width": 4096, "residual": True, "bias": True, "param": "f32"},
        # a small training step of odd sizes, parameters of the activations' type
        {"name": "norm_train_odd", "kind": "norm_train", "dtype": "f16", "rows": 3001,
         "width": 1021, "residual": False, "bias": True, "param": "f16"},
        # 32-bit rows wider than a workgroup's registers are meant for
        {"name": "norm_train_wide", "kind": "norm_train", "dtype": "f32", "rows": 777,
         "width": 20000, "residual": False, "bias": False, "param": "f32"},
        # a training step's recurrence, forward and backward
        {"name": "recur_train", "kind": "recur_train", "dtype": "bf16", "batch": 8,
         "length": 2048, "packed": False, "channels": 4096, "decay": True, "input": True,
         "state": False},
        # one long prompt: one sequence has to fill the chip
        {"name": "recur_long", "kind": "recur", "dtype": "bf16", "batch": 1, "length": 16384,
         "packed": False, "channels": 2048, "decay": True, "input": True, "state": True},
        # packed prompts of different lengths, odd width, continuing from states
        {"name": "recur_packed_odd", "kind": "recur", "dtype": "f16", "batch": 7,
         "length": 701, "packed": True, "channels": 1000, "decay": True, "input": False,
         "state": True},
        # a small 32-bit training step on packed sequences, the plain forget gate
        {"name": "recur_train_odd", "kind": "recur_train", "dtype": "f32", "batch": 3,
         "length": 333, "packed": True, "channels": 520, "decay": False, "input": False,
         "state": True},
        # one token of each sequence of a large serving batch
        {"name": "recur_step", "kind": "recur_step", "dtype": "bf16", "batch": 256,
         "channels": 4096, "decay": True, "input": True},
        # one user's next token, the usual filters: latency
        {"name": "sample_one", "kind": "sample", "dtype": "f32", "rows": 1, "vocab": 50021,
         "settings": "filters", "mask": False},
        # next tokens of a batch without filters: every token's weight counts
        {"name": "sample_all", "kind": "sample", "dtype": "f16", "rows": 64, "vocab": 32000,
         "settings": "temperature", "mask": True},
        # a large serving batch whose users each have settings of their own
        {"name": "sample_batch", "kind": "sample", "dtype": "bf16", "rows": 256,
         "vocab": 131072, "settings": "mixed", "mask": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "norm_train", "norm_train", "recur", "recur", "recur_train",
                       "recur_train", "recur_step", "sample", "sample", "sample"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if kind.startswith("norm"):
        width = rng.choice([_log(rng, 64, 20000), 64 * _log(rng, 1, 256)])
        most = (1 << 27) // _SIZE[dtype] // width  # no more bytes than the training step's
        return {"kind": kind, "dtype": dtype, "rows": _log(rng, 1, min(16384, most)),
                "width": width, "residual": rng.random() < 0.6, "bias": rng.random() < 0.7,
                "param": rng.choice([dtype, "f32"])}
    if kind == "sample":
        vocab = _log(rng, 1000, 131072)
        return {"kind": kind, "dtype": dtype, "rows": _log(rng, 1, 128 if dtype == "f32" else 256),
                "vocab": vocab, "settings": rng.choice(["filters", "temperature", "mixed"]),
                "mask": rng.random() < 0.5}
    channels = rng.choice([_log(rng, 64, 4096), 64 * _log(rng, 1, 64)])
    gates = {"decay": rng.random() < 0.7, "input": rng.random() < 0.6}
    if kind == "recur_step":
        return {"kind": kind, "dtype": dtype, "batch": _log(rng, 1, 256), "channels": channels,
                **gates}
    if dtype == "f32" or kind == "recur":
        channels = min(channels, 2048)
    batch = _log(rng, 1, 16)
    return {"kind": kind, "dtype": dtype, "batch": batch, "length": _log(rng, 1, 16384 // batch),
            "packed": rng.random() < 0.5, "channels": channels, "state": rng.random() < 0.5,
            **gates}


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
    if kind.startswith("norm"):
        r, w, p = case["rows"], case["width"], _SIZE[case["param"]]
        both = 2 if case["residual"] else 1
        params = 1 + int(case["bias"])
        bytes_, flops = 2 * both * r * w * e + params * w * p, 9 * r * w
        if kind == "norm_train":
            # backward: the output's gradient and the input (and the sum's gradient)
            # read, the input's written; the forward pass's input is read again
            bytes_ += (2 + both) * r * w * e + params * w * 4
            flops += 16 * r * w
        return {"bytes": bytes_, "flops": flops}
    if kind == "sample":
        r, v = case["rows"], case["vocab"]
        return {"bytes": r * v * e + 28 * r, "flops": 6 * r * v}
    d = case["channels"]
    ins = 3 if case["input"] else 2
    params = 4 * d if case["decay"] else 0
    if kind == "recur_step":
        b = case["batch"]
        return {"bytes": b * d * (e * (ins + 1) + 8) + params, "flops": 24 * b * d}
    t = case["batch"] * case["length"]
    state = 8 * case["batch"] * d if case["state"] else 0
    if kind == "recur":
        return {"bytes": t * d * e * (ins + 1) + state + params, "flops": 24 * t * d}
    return {"bytes": t * d * e * (2 * ins + 2) + state + 2 * params, "flops": 60 * t * d}


# ------------------------------------------------------------------ the inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = _DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dt=dtype):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dt)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    kind = case["kind"]
    s = {"case": case}
    if kind.startswith("norm"):
        r, w, pt = case["rows"], case["width"], _DTYPES[case["param"]]
        s["x"] = normal(r, w, scale=0.7) if case["residual"] else normal(r, w, scale=2.0)
        s["residual"] = normal(r, w, scale=2.0) if case["residual"] else None
        s["weight"] = (1.0 + 0.2 * normal(w, dt=torch.float32)).to(pt)
        s["bias"] = normal(w, scale=0.1, dt=pt) if case["bias"] else None
        if kind == "norm_train":
            s["dout"] = normal(r, w, scale=0.1)
            s["dsum"] = normal(r, w, scale=0.1) if case["residual"] else None
        return s
    if kind == "sample":
        r, v = case["rows"], case["vocab"]
        x = torch.randn(r, v, generator=gen, device="cuda") * 2.5
        # every other row knows what comes next
        x[::2].scatter_add_(1, torch.randint(v, (r, 1), generator=gen, device="cuda")[::2],
                            torch.full_like(x[::2, :1], 11.0))
        x = x.to(dtype)
        if case["mask"]:  # tokens that a grammar forbids; one row's none is allowed
            x[uniform(r, v) < 0.1] = -math.inf
            x[:, v // 2] = torch.finfo(dtype).min
            if r > 4:
                x[3] = -math.inf
        s["logits"], s["u"] = x, uniform(r)
        if case["settings"] == "temperature":
            s["temperature"], s["top_k"], s["top_p"], s["min_p"] = 0.9, 0, 1.0, 0.0
        elif case["settings"] == "filters":
            s["temperature"], s["top_k"], s["top_p"], s["min_p"] = 0.8, 50, 0.95, 0.0
        else:
            def pick(values, dt):
                at = torch.randint(len(values), (r,), generator=gen, device="cuda")
                return torch.tensor(values, dtype=dt, device="cuda")[at]

            f = torch.float32
            s["temperature"] = pick([0.0, 0.6, 0.8, 1.0, 1.0, 1.3], f)
            s["top_k"] = pick([0, 0, 1, 20, 50, 200, 5000], torch.int32)
            s["top_p"] = pick([1.0, 1.0, 0.5, 0.9, 0.95], f)
            s["min_p"] = pick([0.0, 0.0, 0.02, 0.1], f)
        return s
    d, f32 = case["channels"], torch.float32
    s["decay"] = None
    if case["decay"]:  # a between 0.9 and 0.999 at an open gate
        s["decay"] = -torch.log(0.9 + 0.099 * uniform(d))
    if kind == "recur_step":
        b = case["batch"]
        s["x"], s["gate"] = normal(b, d), normal(b, d)
        s["input_gate"] = normal(b, d) if case["input"] else None
        s["state"] = normal(b, d, scale=0.5, dt=f32)
        return s
    b = case["batch"]
    lens = _lengths(case)
    lead = (sum(lens),) if case["packed"] else (b, case["length"])
    s["lens"], s["starts"] = lens, None
    if case["packed"]:
        s["starts"] = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
    s["x"], s["gate"] = normal(*lead, d), normal(*lead, d)
    s["input_gate"] = normal(*lead, d) if case["input"] else None
    s["init_state"] = normal(b, d, scale=0.5, dt=f32) if case["state"] else None
    train = kind == "recur_train"
    s["final_state"] = (torch.empty(b, d, dtype=f32, device="cuda")
                        if case["state"] and not train else None)
    if train:
        s["dout"] = normal(*lead, d)
    return s


# ------------------------------------------------------------- the library's calls
def _run_own(s):
    import scan_canonical_reduce_amd as canon

    case = s["case"]
    kind = case["kind"]
    if kind.startswith("norm"):
        x, w, b = s["x"], s["weight"], s["bias"]
        stats = canon.layer_norm_stats(x) if kind == "norm_train" else None
        if case["residual"]:
            out, total = canon.add_layer_norm(x, s["residual"], w, b, _EPS, stats=stats)
            res = (out, total)
        else:
            total = x
            res = (canon.layer_norm(x, w, b, _EPS, stats=stats),)
        if kind == "norm":
            return res
        g = canon.layer_norm_grad(s["dout"], total, w, stats, bias=b, dsum=s["dsum"])
        return res + (g.dx, g.dweight) + ((g.dbias,) if case["bias"] else ())
    if kind == "sample":
        return canon.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"],
                            top_p=s["top_p"], min_p=s["min_p"])
    gates = dict(decay=s["decay"], input_gate=s["input_gate"])
    if kind == "recur_step":
        nxt = torch.empty_like(s["state"])
        out = canon.gated_recurrence_step(s["state"], s["x"], s["gate"], out_state=nxt, **gates)
        return out, nxt
    if kind == "recur":
        out = canon.gated_recurrence(s["x"], s["gate"], starts=s["starts"],
                                     init_state=s["init_state"], final_state=s["final_state"],
                                     **gates)
        return (out, s["final_state"]) if case["state"] else (out,)
    states = canon.gated_recurrence_states(s["x"], s["starts"])
    out = canon.gated_recurrence(s["x"], s["gate"], starts=s["starts"],
                                 init_state=s["init_state"], states=states, **gates)
    g = canon.gated_recurrence_grad(s["dout"], s["x"], s["gate"], states, starts=s["starts"],
                                    **gates)
    return ((out, g.dx, g.dgate) + ((g.ddecay,) if case["decay"] else ())
            + ((g.dinput_gate,) if case["input"] else ())
            + ((g.dinit_state,) if case["state"] else ()))


# ---------------------------------------------------------------- the plain forms
def _norm_plain(s):
    case = s["case"]
    dtype = s["x"].dtype
    res = ()
    x = s["x"]
    if case["residual"]:
        x = (x.float() + s["residual"].float()).to(dtype)
        res = (x,)
    x, w = x.float(), s["weight"].float()
    centred = x - x.mean(-1, keepdim=True)
    rstd = torch.rsqrt((centred * centred).mean(-1, keepdim=True) + _EPS)
    unit = centred * rstd
    out = unit * w
    if case["bias"]:
        out = out + s["bias"].float()
    res = (out.to(dtype),) + res
    if case["kind"] == "norm":
        return res
    dout = s["dout"].float()
    g = dout * w
    dx = rstd * (g - g.mean(-1, keepdim=True) - unit * (g * unit).mean(-1, keepdim=True))
    if case["residual"]:
        dx = dx + s["dsum"].float()
    res += (dx.to(dtype), (dout * unit).sum(0))
    return res + ((dout.sum(0),) if case["bias"] else ())


def _sample_plain(s):
    x, rows = s["logits"], s["case"]["rows"]

    def per_row(v):
        return v.double()[:, None] if torch.is_tensor(v) else x.new_full((rows, 1), v,
                                                                         dtype=torch.float64)

    order = torch.sort(x.float(), dim=1, descending=True, stable=True)[1]
    best = x.gather(1, order[:, :1])
    temp, k = per_row(s["temperature"]), per_row(s["top_k"])
    p, least = per_row(s["top_p"]), per_row(s["min_p"])
    w = torch.exp((x.double() - best.double()) / torch.where(temp > 0, temp, 1.0))
    w = torch.where(x == best, torch.ones_like(w), w)
    ranked = w.gather(1, order)
    place = torch.arange(x.shape[1], device=x.device)
    ranked = ranked * ((k <= 0) | (place < k))
    before = torch.cumsum(ranked, 1) - ranked
    keep = (p >= 1) | (place == 0) | (before < p * ranked.sum(1, keepdim=True))
    ranked = ranked * (keep & (ranked >= least))
    w = torch.zeros_like(w).scatter_(1, order, ranked)
    total = torch.cumsum(w, 1)
    got = (total > s["u"].double()[:, None] * total[:, -1:]) & (w > 0)
    # beyond the last border by rounding: the last token with a weight
    last = torch.where(w > 0, place, -1).amax(1)
    ids = torch.where(got.any(1), got.to(torch.uint8).argmax(1), last)
    ids = torch.where(temp[:, 0] > 0, ids, order[:, 0])
    return torch.where(best[:, 0] == -math.inf, -1, ids)


def _pad(x, s):
    """[sequences, longest, channels] in 64 bits, packed sequences padded with 0."""
    if s["starts"] is None:
        return x.double()
    out = x.new_zeros((len(s["lens"]), max(s["lens"]), x.shape[-1]), dtype=torch.float64)
    at = 0
    for i, n in enumerate(s["lens"]):
        out[i, :n] = x[at:at + n]
        at += n
    return out


def _unpad(x, s, dtype):
    if s["starts"] is None:
        return x.to(dtype)
    return torch.cat([x[i, :n] for i, n in enumerate(s["lens"])]).to(dtype)


def _gates_plain(s, gate, input_gate):
    """a, the factor of x before the input gate, the input gate, and sigmoid(gate)"""
    r = torch.sigmoid(gate)
    i = 1.0 if input_gate is None else torch.sigmoid(input_gate)
    if s["decay"] is None:
        return r, torch.sigmoid(-gate), i, r
    log_a = -s["decay"] * r
    return torch.exp(log_a), torch.sqrt(-torch.expm1(2.0 * log_a)), i, r


def _recur_plain(s, backward):
    case, dtype = s["case"], s["x"].dtype
    x = _pad(s["x"], s)
    gate = _pad(s["gate"], s)
    inp = _pad(s["input_gate"], s) if case["input"] else None
    a, c, i, r = _gates_plain(s, gate, inp)
    n, length, d = x.shape
    if s["starts"] is not None:  # padding leaves the state as it is
        ends = torch.tensor(s["lens"], device=x.device)[:, None]
        inside = (torch.arange(length, device=x.device) < ends)[..., None]
        a, c = torch.where(inside, a, 1.0), torch.where(inside, c, 0.0)
    at = a.transpose(0, 1).contiguous()
    h = torch.empty(length + 1, n, d, dtype=x.dtype, device=x.device)
    h[1:] = (c * i * x).transpose(0, 1)
    h[0] = s["init_state"] if s["init_state"] is not None else 0.0
    for t in range(length):
        h[t + 1].addcmul_(at[t], h[t])
    out = _unpad(h[1:].transpose(0, 1), s, dtype)
    if not backward:
        return (out, h[length].float()) if case["state"] else (out,)
    lam = _pad(s["dout"], s).transpose(0, 1).contiguous()
    for t in range(length - 1, 0, -1):
        lam[t - 1].addcmul_(at[t], lam[t])
    dinit = at[0] * lam[0]
    lam, prev = lam.transpose(0, 1), h[:length].transpose(0, 1)
    dx = lam * c * i
    res = (out, _unpad(dx, s, dtype))
    if s["decay"] is None:
        dgate = lam * (prev - i * x) * a * c
        res += (_unpad(dgate, s, dtype),)
    else:
        slope = torch.where(c > 0, a * a / torch.where(c > 0, c, 1.0), 0.0)
        dlog = lam * (a * prev - slope * i * x)
        if s["starts"] is not None:
            dlog = dlog * inside
        res += (_unpad(-s["decay"] * dlog * r * (1.0 - r), s, dtype),
                -(dlog * r).sum((0, 1)).float())
    if case["input"]:
        res += (_unpad(lam * c * x * i * (1.0 - i), s, dtype),)
    return res + ((dinit.float(),) if case["state"] else ())


def run(s):
    if own:
        return _run_own(s)
    kind = s["case"]["kind"]
    if kind.startswith("norm"):
        return _norm_plain(s)
    if kind == "sample":
        return _sample_plain(s)
    if kind == "recur_step":
        x = s["x"].float()
        inp = s["input_gate"].float() if s["case"]["input"] else None
        a, c, i, _ = _gates_plain(s, s["gate"].float(), inp)
        h = a * s["state"] + c * i * x
        return h.to(s["x"].dtype), h
    return _recur_plain(s, kind == "recur_train")


# ------------------------------------------------------------------------- exact
def _exact_norm(s):
    case = s["case"]
    dtype, n = s["x"].dtype, case["width"]
    outs, sums, dxs = [], [], []
    w = s["weight"].double()
    dw, db = torch.zeros_like(w), torch.zeros_like(w)
    step = max(1, (1 << 26) // n)
    for lo in range(0, case["rows"], step):
        rows = slice(lo, lo + step)
        x = s["x"][rows]
        if case["residual"]:
            sums.append(x.double() + s["residual"][rows].double())
            x = (x.float() + s["residual"][rows].float()).to(dtype)  # as it is stored
        x = x.double()
        mean = x.sum(1, keepdim=True) / n
        var = (x * x).sum(1, keepdim=True) / n - mean * mean
        std = torch.sqrt(var + _EPS)
        unit = (x - mean) / std
        outs.append(unit * w + (s["bias"].double() if case["bias"] else 0.0))
        if case["kind"] == "norm":
            continue
        dout = s["dout"][rows].double()
        dw += (dout * unit).sum(0)
        db += dout.sum(0)
        dunit = dout * w
        dvar = (dunit * (x - mean)).sum(1, keepdim=True) * -0.5 / std ** 3
        dmean = -(dunit / std).sum(1, keepdim=True)
        dx = dunit / std + dvar * 2.0 * (x - mean) / n + dmean / n
        dxs.append(dx + (s["dsum"][rows].double() if case["residual"] else 0.0))
    res = (torch.cat(outs),) + ((torch.cat(sums),) if case["residual"] else ())
    if case["kind"] == "norm":
        return res
    return res + (torch.cat(dxs), dw) + ((db,) if case["bias"] else ())


def _exact_sample(s):
    case = s["case"]
    rows = case["rows"]

    def per_row(v):
        return v.tolist() if torch.is_tensor(v) else [v] * rows

    u, temps, ks = s["u"].tolist(), per_row(s["temperature"]), per_row(s["top_k"])
    ps, leasts = per_row(s["top_p"]), per_row(s["min_p"])
    ids = []
    for i in range(rows):
        x = s["logits"][i].double().cpu().numpy()
        order = np.lexsort((np.arange(x.size), -x))  # largest first, then lowest index
        if x[order[0]] == -math.inf:
            ids.append(-1)
            continue
        if temps[i] == 0:
            ids.append(int(order[0]))
            continue
        if ks[i] > 0:
            order = order[:ks[i]]
        w = np.exp((x[order] - x[order[0]]).astype(np.longdouble) / np.longdouble(temps[i]))
        if ps[i] < 1:
            total = np.cumsum(w)
            order = order[:1 + int(np.searchsorted(total, np.longdouble(ps[i]) * total[-1]))]
            w = w[:order.size]
        allowed = w >= leasts[i]
        order, w = order[allowed], w[allowed]
        by_index = np.argsort(order)
        order, total = order[by_index], np.cumsum(w[by_index])
        at = int(np.searchsorted(total, np.longdouble(u[i]) * total[-1], side="right"))
        ids.append(int(order[min(at, order.size - 1)]))
    return torch.tensor(ids, device="cuda")


def _fold64(a, b, h0):
    """h[t] = a[t] h[t-1] + b[t] along dimension 0, by doubling; destroys a and b."""
    b[0] += a[0] * h0
    n, step = a.shape[0], 1
    while step < n:
        b[step:] += a[step:] * b[:-step].clone()
        a[step:] *= a[:-step].clone()
        step *= 2
    return b


def _exact_recur(s, backward):
    case = s["case"]
    d, shape = case["channels"], s["x"].shape
    total, dev = s["x"].numel() // d, s["x"].device

    def flat(name):
        return None if s[name] is None else s[name].reshape(-1, d)

    def new(*size):
        return torch.zeros(*size, dtype=torch.float64, device=dev)

    x, gate, inp = flat("x"), flat("gate"), flat("input_gate")
    dout = flat("dout") if backward else None
    out, final = new(total, d), new(case["batch"], d)
    if backward:
        dx, dgate, dinp = new(total, d), new(total, d), new(total, d)
        ddecay, dinit = new(d), new(case["batch"], d)
    at = 0
    for k, length in enumerate(s["lens"]):
        rows = slice(at, at + length)
        at += length
        h0 = s["init_state"][k].double() if s["init_state"] is not None else new(d)
        if length == 0:
            final[k] = h0
            continue
        z, xs = gate[rows].double(), x[rows].double()
        r = 1.0 / (1.0 + torch.exp(-z))
        i = 1.0 / (1.0 + torch.exp(-inp[rows].double())) if case["input"] else torch.ones_like(r)
        if case["decay"]:
            D = s["decay"].double()
            a = torch.exp(-D * r)
            c = torch.sqrt(-torch.expm1(-2.0 * D * r))
        else:
            a, c = r, 1.0 / (1.0 + torch.exp(z))
        h = _fold64(a.clone(), c * i * xs, h0)
        out[rows], final[k] = h, h[-1]
        if not backward:
            continue
        later = torch.cat([torch.zeros_like(a[:1]), a[1:].flip(0)])
        lam = _fold64(later, dout[rows].double().flip(0), torch.zeros_like(h0)).flip(0)
        dinit[k] = a[0] * lam[0]
        da = lam * torch.cat([h0[None], h[:-1]])
        dc = lam * i * xs
        dx[rows] = lam * c * i
        dinp[rows] = lam * c * xs * i * (1.0 - i)
        if case["decay"]:
            # da/dr = -D a, dc/dr = D a^2 / c, and the same over D for r
            both = a * a / c * dc - a * da
            dgate[rows] = both * D * r * (1.0 - r)
            ddecay += (both * r).sum(0)
        else:
            dgate[rows] = (da - dc) * r * c
    if not backward:
        return (out.view(shape), final) if case["state"] else (out.view(shape),)
    return ((out.view(shape), dx.view(shape), dgate.view(shape))
            + ((ddecay,) if case["decay"] else ())
            + ((dinp.view(shape),) if case["input"] else ())
            + ((dinit,) if case["state"] else ()))


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind.startswith("norm"):
        return _exact_norm(s)
    if kind == "sample":
        return _exact_sample(s)
    if kind == "recur_step":
        x, z = s["x"].double(), s["gate"].double()
        r = 1.0 / (1.0 + torch.exp(-z))
        if case["decay"]:
            log_a = -s["decay"].double() * r
            a, c = torch.exp(log_a), torch.sqrt(-torch.expm1(2.0 * log_a))
        else:
            a, c = r, 1.0 - r
        if case["input"]:
            c = c / (1.0 + torch.exp(-s["input_gate"].double()))
        h = a * s["state"].double() + c * x
        return h, h
    return _exact_recur(s, kind == "recur_train")
