"""Operators of a recurrent language model's layers: layer norm with the residual
sum, the gated linear recurrence, and sampling of the next token.

Argument marshalling only, as in the package itself; the C ABI is declared in
``include/canon_layer.h``, which states what each operator computes.  Shapes,
types, streams and workspaces are those of the sequence operators (``seq.py``).
"""
from __future__ import annotations

import ctypes
import operator
import struct
from typing import NamedTuple, Optional

import torch

from . import CanonError, lib
from .seq import (DTYPES, _NONE, _call, _dtype, _flat, _rows, _same, _sequences, _step_rows,
                  _workspace)

LAYER_VERSION = 1

LAYER_EXPORTS = [
    "canon_layer_version", "canon_layer_norm", "canon_layer_norm_grad_workspace_bytes",
    "canon_layer_norm_grad", "canon_gated_recurrence_states",
    "canon_gated_recurrence_workspace_bytes", "canon_gated_recurrence",
    "canon_gated_recurrence_grad_workspace_bytes", "canon_gated_recurrence_grad",
    "canon_gated_recurrence_step", "canon_sample_workspace_bytes", "canon_sample",
]

# canon_norm_t, canon_recur_t and canon_sample_t: fields of 8 bytes, doubles among them
NORM = struct.Struct("=5qd26q")
RECUR = struct.Struct("=36q")
SAMPLE = struct.Struct("=10q3d3q")

_layer = None


def _lib() -> ctypes.CDLL:
    global _layer
    if _layer is not None:
        return _layer
    L = lib()
    S, I, P = ctypes.c_size_t, ctypes.c_int, ctypes.c_void_p
    for name in LAYER_EXPORTS:
        f = getattr(L, name)
        f.restype = S if name.endswith("_bytes") or name.endswith("_states") else I
    L.canon_layer_norm.argtypes = [P, P]
    L.canon_layer_norm_grad_workspace_bytes.argtypes = [S, S, S]
    L.canon_layer_norm_grad.argtypes = [P, P, S, P]
    L.canon_gated_recurrence_states.argtypes = [S, S, I, S]
    L.canon_gated_recurrence_workspace_bytes.argtypes = [S, S, I, S]
    L.canon_gated_recurrence.argtypes = [P, P, S, P]
    L.canon_gated_recurrence_grad_workspace_bytes.argtypes = [S, S, I, S]
    L.canon_gated_recurrence_grad.argtypes = [P, P, S, P]
    L.canon_gated_recurrence_step.argtypes = [P, P]
    L.canon_sample_workspace_bytes.argtypes = [S, S]
    L.canon_sample.argtypes = [P, P, S, P]
    if L.canon_layer_version() != LAYER_VERSION:
        raise CanonError("libcanon layer operators: version mismatch")
    _layer = L
    return L


def _new(x: torch.Tensor) -> torch.Tensor:
    """A contiguous uninitialised tensor like x (empty_like takes half a microsecond less
    than new_empty, a twentieth of a small call)."""
    return torch.empty_like(x) if x.is_contiguous() else x.new_empty(x.shape)


def _new_rows(t: torch.Tensor, shape, lead: int):
    """canon_rows_t of what _new gave: nothing to check."""
    width = shape[-1]
    return t.data_ptr(), shape[1] * width if lead == 2 else 0, width


# ------------------------------------------------------------------ layer norm
class LayerNormGrads(NamedTuple):
    dx: torch.Tensor
    dweight: torch.Tensor
    dbias: Optional[torch.Tensor]


def _norm(what, x, weight, bias):
    """(dtype, param_dtype, seqs, rows, width), leading dimensions, (weight, bias)"""
    d = _dtype(x, what)
    if x.dim() not in (2, 3):
        raise ValueError(f"{what} takes [rows, width] or [sequences, rows, width]")
    width = x.shape[-1]
    if weight.dtype != x.dtype and weight.dtype != torch.float32:
        raise TypeError(f"{what}: weight must be {x.dtype} or float32, not {weight.dtype}")
    seqs = x.shape[0] if x.dim() == 3 else 1
    head = (d, DTYPES[weight.dtype], seqs, x.shape[-2], width)
    return head, x.dim() - 1, (_flat(what, "weight", weight, (width,), weight.dtype),
                               _flat(what, "bias", bias, (width,), weight.dtype))


def layer_norm_stats(x: torch.Tensor) -> torch.Tensor:
    """An uninitialised buffer for the `stats` of layer_norm of x: each row's mean
    and 1 / standard deviation, for the backward pass."""
    return torch.empty((*x.shape[:-1], 2), dtype=torch.float32, device=x.device)


def _layer_norm(what, x, residual, weight, bias, eps, stats, total, out):
    _same(what, x.device, residual, weight, bias, stats, total, out)
    head, lead, params = _norm(what, x, weight, bias)
    shape, dtype = x.shape, x.dtype
    if out is None:
        out = _new(x)
        o = _new_rows(out, shape, lead)
    else:
        o = _rows(what, "out", out, shape, dtype, lead)
    r = t = _NONE
    if residual is not None:
        r = _rows(what, "residual", residual, shape, dtype, lead)
        if total is None:
            total = _new(x)
            t = _new_rows(total, shape, lead)
        else:
            t = _rows(what, "sum_out", total, shape, dtype, lead)
    c = NORM.pack(*head, eps, *_rows(what, "x", x, shape, dtype, lead), *r, *t, *o, *params,
                  _flat(what, "stats", stats, (*shape[:lead], 2), torch.float32) if stats is not None
                  else 0, *_NONE, *_NONE, *_NONE, 0, 0)
    _call(what, x.device, _lib().canon_layer_norm, c)
    return out, total


def layer_norm(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
               eps: float = 1e-5, stats: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Each row of x ([rows, width] or [sequences, rows, width], any row and sequence
    strides) less its mean, over its standard deviation, times weight, plus bias
    (float32 or x's type).  stats: a buffer of layer_norm_stats that is written for
    layer_norm_grad.  out may be x."""
    return _layer_norm("layer_norm", x, None, weight, bias, eps, stats, None, out)[0]


def add_layer_norm(x: torch.Tensor, residual: torch.Tensor, weight: torch.Tensor,
                   bias: Optional[torch.Tensor] = None, eps: float = 1e-5,
                   stats: Optional[torch.Tensor] = None, sum_out: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None) -> tuple[torch.Tensor, torch.Tensor]:
    """(layer_norm(s, ...), s) with s = x + residual, rounded to their type, in one
    pass.  sum_out and out may each be x or residual (not the same one)."""
    return _layer_norm("add_layer_norm", x, residual, weight, bias, eps, stats, sum_out, out)


def layer_norm_grad_workspace_bytes(seqs: int, rows: int, width: int) -> int:
    return _lib().canon_layer_norm_grad_workspace_bytes(seqs, rows, width)


def layer_norm_grad(dout: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                    stats: torch.Tensor, bias: Optional[torch.Tensor] = None,
                    dsum: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                    ws: Optional[torch.Tensor] = None) -> LayerNormGrads:
    """Gradients of layer_norm's inputs, given the `stats` that its call wrote; of
    add_layer_norm's with x = its sum, whose own gradient dsum is added (dx is then
    the gradient of both addends).  dweight and dbias (with bias) are float32.  dx may
    be dout or dsum."""
    what = "layer_norm_grad"
    _same(what, x.device, dout, weight, stats, bias, dsum, dx, ws)
    head, lead, params = _norm(what, x, weight, bias)
    shape, dtype, device = x.shape, x.dtype, x.device
    if dx is None:
        dx = _new(x)
        d = _new_rows(dx, shape, lead)
    else:
        d = _rows(what, "dx", dx, shape, dtype, lead)
    dw = torch.empty(head[4], dtype=torch.float32, device=device)
    db = None if bias is None else torch.empty(head[4], dtype=torch.float32, device=device)
    c = NORM.pack(*head, 0.0, *_rows(what, "x", x, shape, dtype, lead), *_NONE, *_NONE, *_NONE,
                  *params, _flat(what, "stats", stats, (*shape[:lead], 2), torch.float32),
                  *_rows(what, "dout", dout, shape, dtype, lead),
                  *(_NONE if dsum is None else _rows(what, "dsum", dsum, shape, dtype, lead)),
                  *d, dw.data_ptr(),
                  0 if db is None else db.data_ptr())
    L = _lib()
    w = _workspace(L.canon_layer_norm_grad_workspace_bytes(*head[2:5]), device, ws)
    _call(what, device, L.canon_layer_norm_grad, c, w.data_ptr(), w.numel())
    return LayerNormGrads(dx, dw, db)


# ------------------------------------------------------ gated linear recurrence
class GatedRecurrenceGrads(NamedTuple):
    dx: torch.Tensor
    dgate: torch.Tensor
    ddecay: Optional[torch.Tensor]
    dinput_gate: Optional[torch.Tensor]
    dinit_state: torch.Tensor


def gated_recurrence_workspace_bytes(seqs: int, rows: int, packed: bool, channels: int) -> int:
    return _lib().canon_gated_recurrence_workspace_bytes(seqs, rows, int(packed), channels)


def gated_recurrence_grad_workspace_bytes(seqs: int, rows: int, packed: bool,
                                          channels: int) -> int:
    return _lib().canon_gated_recurrence_grad_workspace_bytes(seqs, rows, int(packed), channels)


def gated_recurrence_states(x: torch.Tensor,
                            starts: Optional[torch.Tensor] = None) -> torch.Tensor:
    """An uninitialised buffer for gated_recurrence's `states` argument: what the
    forward pass of x saves for the backward pass (4 bytes per 128 elements of x)."""
    seqs, rows, _, lead = _sequences("gated_recurrence_states", x, starts)
    n = _lib().canon_gated_recurrence_states(seqs, rows, int(lead == 1), x.shape[-1])
    return torch.empty(n, dtype=torch.float32, device=x.device)


def gated_recurrence(x: torch.Tensor, gate: torch.Tensor, decay: Optional[torch.Tensor] = None,
                     input_gate: Optional[torch.Tensor] = None,
                     starts: Optional[torch.Tensor] = None,
                     init_state: Optional[torch.Tensor] = None,
                     final_state: Optional[torch.Tensor] = None,
                     states: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                     ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """h[t] = a h[t-1] + c i x[t] over the rows of each sequence, channel by channel:
    a = exp(-decay sigmoid(gate)) and c = sqrt(1 - a^2), or without decay
    a = sigmoid(gate) and c = 1 - a; i = sigmoid(input_gate), or 1 without.

    x, gate, input_gate: activations of one shape; decay [channels] float32, finite, not
    negative.  init_state, final_state [sequences, channels] float32: h before the
    first row and after the last (written, and may be init_state).  states: a buffer of
    gated_recurrence_states for the backward pass."""
    what = "gated_recurrence"
    _same(what, x.device, gate, decay, input_gate, starts, init_state, final_state, states, out, ws)
    seqs, rows, sp, lead = _sequences(what, x, starts)
    shape, dtype, f32, channels = x.shape, x.dtype, torch.float32, x.shape[-1]
    packed = int(lead == 1)
    L = _lib()
    kept = 0
    if states is not None:
        kept = _flat(what, "states", states,
                     (L.canon_gated_recurrence_states(seqs, rows, packed, channels),), f32)
    d = _dtype(x, what)
    if out is None:
        out = _new(x)
        o = _new_rows(out, shape, lead)
    else:
        o = _rows(what, "out", out, shape, dtype, lead)
    state = (seqs, channels)
    c = RECUR.pack(d, seqs, rows, channels, sp, *_rows(what, "x", x, shape, dtype, lead),
                   *_rows(what, "gate", gate, shape, dtype, lead),
                   *(_NONE if input_gate is None else
                     _rows(what, "input_gate", input_gate, shape, dtype, lead)), *o,
                   _flat(what, "decay", decay, (channels,), f32),
                   _flat(what, "init_state", init_state, state, f32),
                   _flat(what, "final_state", final_state, state, f32), kept,
                   *_NONE, *_NONE, *_NONE, *_NONE, 0, 0, 0)
    w = _workspace(L.canon_gated_recurrence_workspace_bytes(seqs, rows, packed, channels),
                   x.device, ws)
    _call(what, x.device, L.canon_gated_recurrence, c, w.data_ptr(), w.numel())
    return out


def gated_recurrence_grad(dout: torch.Tensor, x: torch.Tensor, gate: torch.Tensor,
                          states: torch.Tensor, decay: Optional[torch.Tensor] = None,
                          input_gate: Optional[torch.Tensor] = None,
                          starts: Optional[torch.Tensor] = None,
                          d_final_state: Optional[torch.Tensor] = None,
                          ws: Optional[torch.Tensor] = None) -> GatedRecurrenceGrads:
    """Gradients of gated_recurrence's inputs, given the `states` that its call with
    these inputs wrote, and the gradients of its output and (optionally) final state.
    Activations' gradients have their type, the others are float32; rows that belong to
    no sequence have undefined gradients."""
    what = "gated_recurrence_grad"
    _same(what, x.device, dout, gate, states, decay, input_gate, starts, d_final_state, ws)
    seqs, rows, sp, lead = _sequences(what, x, starts)
    shape, dtype, f32, channels = x.shape, x.dtype, torch.float32, x.shape[-1]
    packed, device = int(lead == 1), x.device
    L = _lib()
    size = L.canon_gated_recurrence_states(seqs, rows, packed, channels)
    d = _dtype(x, what)

    def empty(*s):
        return torch.empty(s, dtype=f32, device=device)

    g = GatedRecurrenceGrads(
        dx=_new(x), dgate=_new(x),
        ddecay=None if decay is None else empty(channels),
        dinput_gate=None if input_gate is None else _new(x),
        dinit_state=empty(seqs, channels))
    gi = _NONE, _NONE
    if input_gate is not None:
        gi = (_rows(what, "input_gate", input_gate, shape, dtype, lead),
              _new_rows(g.dinput_gate, shape, lead))
    c = RECUR.pack(d, seqs, rows, channels, sp, *_rows(what, "x", x, shape, dtype, lead),
                   *_rows(what, "gate", gate, shape, dtype, lead), *gi[0], *_NONE,
                   _flat(what, "decay", decay, (channels,), f32), 0, 0,
                   _flat(what, "states", states, (size,), f32),
                   *_rows(what, "dout", dout, shape, dtype, lead),
                   *_new_rows(g.dx, shape, lead), *_new_rows(g.dgate, shape, lead), *gi[1],
                   0 if decay is None else g.ddecay.data_ptr(),
                   _flat(what, "d_final_state", d_final_state, (seqs, channels), f32),
                   g.dinit_state.data_ptr())
    w = _workspace(L.canon_gated_recurrence_grad_workspace_bytes(seqs, rows, packed, channels),
                   device, ws)
    _call(what, device, L.canon_gated_recurrence_grad, c, w.data_ptr(), w.numel())
    return g


def gated_recurrence_step(state: torch.Tensor, x: torch.Tensor, gate: torch.Tensor,
                          decay: Optional[torch.Tensor] = None,
                          input_gate: Optional[torch.Tensor] = None,
                          out_state: Optional[torch.Tensor] = None,
                          out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """gated_recurrence for one row of each sequence: x, gate, input_gate [sequences,
    channels].  The state [sequences, channels] is updated in place, or, with
    out_state, read and written there.  out may be x or a gate."""
    what = "gated_recurrence_step"
    _same(what, x.device, state, gate, decay, input_gate, out_state, out)
    if x.dim() != 2:
        raise ValueError(f"{what} takes [sequences, channels]")
    shape, dtype, f32 = x.shape, x.dtype, torch.float32
    d = _dtype(x, what)
    old = _flat(what, "state", state, shape, f32)
    if out is None:
        out = _new(x)
        o = out.data_ptr(), shape[1], 0
    else:
        o = _step_rows(what, "out", out, shape, dtype)
    c = RECUR.pack(d, shape[0], 1, shape[1], 0, *_step_rows(what, "x", x, shape, dtype),
                   *_step_rows(what, "gate", gate, shape, dtype),
                   *(_NONE if input_gate is None else
                     _step_rows(what, "input_gate", input_gate, shape, dtype)),
                   *o, _flat(what, "decay", decay, shape[1:], f32), old,
                   old if out_state is None else _flat(what, "out_state", out_state, shape, f32),
                   0, *_NONE, *_NONE, *_NONE, *_NONE, 0, 0, 0)
    _call(what, x.device, _lib().canon_gated_recurrence_step, c)
    return out


# -------------------------------------------------------------------- sampling
def _setting(what: str, name: str, v, rows: int, dtype: torch.dtype):
    """(pointer, value) of a number for all rows, or one per row"""
    if not torch.is_tensor(v):
        if dtype == torch.int32:
            try:
                v = operator.index(v)
            except TypeError:
                raise TypeError(f"{what}: {name} must be an integer, not {v!r}") from None
        return 0, v
    return _flat(what, name, v, (rows,), dtype), 0


def sample_workspace_bytes(rows: int, vocab: int) -> int:
    return _lib().canon_sample_workspace_bytes(rows, vocab)


def sample(logits: torch.Tensor, u: torch.Tensor, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0,
           out: Optional[torch.Tensor] = None,
           ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token of each row of logits ([rows, vocab], any row stride), int64 (or out's
    int32): the softmax of logits / temperature, cut to the top_k largest, of those to
    the fewest largest that have top_p of the sum, of those to the ones with at least
    min_p times the largest's weight; the token at which the sum in index order passes
    u (float32 [rows], in [0, 1)) times the whole.

    Each setting is a number or a tensor of one per row (float32; top_k int32).  A
    temperature of 0 takes the largest logit; top_k of 0, top_p of 1 and min_p of 0 keep
    everything.  Ties go to the lowest index.  Logits of minus infinity and NaN are
    never taken; a row of nothing else gives -1."""
    what = "sample"
    given = [t for t in (temperature, top_k, top_p, min_p) if torch.is_tensor(t)]
    _same(what, logits.device, u, out, ws, *given)
    d = _dtype(logits, what)
    if logits.dim() != 2 or (logits.shape[1] > 1 and logits.numel() and logits.stride(1) != 1):
        raise ValueError(f"{what}: logits must be 2-d with unit column stride")
    rows, vocab = logits.shape
    f32, i32 = torch.float32, torch.int32
    tp, tv = _setting(what, "temperature", temperature, rows, f32)
    kp, kv = _setting(what, "top_k", top_k, rows, i32)
    pp, pv = _setting(what, "top_p", top_p, rows, f32)
    mp, mv = _setting(what, "min_p", min_p, rows, f32)
    if tv < 0 or kv < 0 or not 0 <= pv <= 1 or not 0 <= mv <= 1 or tv != tv:
        raise ValueError(f"{what}: temperature and top_k must not be negative, top_p and min_p "
                         "lie in [0, 1]")
    kv = min(kv, vocab)  # no more than there are
    if out is None:
        out = torch.empty(rows, dtype=torch.int64, device=logits.device)
    elif out.dtype not in (torch.int64, i32):
        raise TypeError(f"{what}: out must be int64 or int32, not {out.dtype}")
    c = SAMPLE.pack(d, rows, vocab, logits.data_ptr(), logits.stride(0) if rows > 1 else 0,
                    _flat(what, "u", u, (rows,), f32), tp, kp, pp, mp, tv, pv, mv, kv,
                    _flat(what, "out", out, (rows,), out.dtype), out.element_size())
    L = _lib()
    w = _workspace(L.canon_sample_workspace_bytes(rows, vocab), logits.device, ws)
    _call(what, logits.device, L.canon_sample, c, w.data_ptr(), w.numel())
    return out
