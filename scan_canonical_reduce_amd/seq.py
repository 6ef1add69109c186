"""Operators of sequence models: embedding, causal convolution, selective scan.

Argument marshalling only, as in the package itself; the C ABI is declared in
``include/canon_seq.h``, which states what each operator computes.

Shapes.  Activations (float32, bfloat16 or float16, one type per call) are
``[sequences, rows, columns]``, or with ``starts`` (int32, sequences + 1
ascending row offsets, on the GPU) ``[rows, columns]`` with the sequences
packed one after the other; rows outside them are left as they are.  Columns
have unit stride, rows and sequences any.  Parameters, their gradients and scan
states are float32 and contiguous.

Calls run on the current stream of the tensors' device.  ``ws`` is a
caller-owned uint8 workspace of ``*_workspace_bytes(...)`` bytes; without it,
or if it is too small, the call allocates its own.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import CanonError, _check, lib

DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
CONV_CHUNK = 32
SCAN_CHUNK = 64
MAX_STATES = 16
MAX_TAPS = 8
SEQ_VERSION = 1

SEQ_EXPORTS = [
    "canon_seq_version", "canon_embedding", "canon_embedding_grad_workspace_bytes",
    "canon_embedding_grad", "canon_causal_conv", "canon_causal_conv_grad_workspace_bytes",
    "canon_causal_conv_grad", "canon_causal_conv_step", "canon_selective_scan_states",
    "canon_selective_scan_workspace_bytes", "canon_selective_scan",
    "canon_selective_scan_grad_workspace_bytes", "canon_selective_scan_grad",
    "canon_selective_scan_step",
]

_I64, _P = ctypes.c_int64, ctypes.c_void_p


class Rows(ctypes.Structure):
    """canon_rows_t"""
    _fields_ = [("p", _P), ("seq", _I64), ("row", _I64)]


class Conv(ctypes.Structure):
    """canon_conv_t"""
    _fields_ = [(n, _I64) for n in
                ("dtype", "taps", "silu", "param_dtype", "seqs", "rows", "channels")] + [
        ("starts", _P), ("x", Rows), ("out", Rows), ("weight", _P), ("bias", _P),
        ("init_state", _P), ("final_state", _P), ("dout", Rows), ("dx", Rows), ("dweight", _P),
        ("dbias", _P), ("d_final_state", _P), ("d_init_state", _P)]


class Scan(ctypes.Structure):
    """canon_selective_scan_t"""
    _fields_ = [(n, _I64) for n in
                ("dtype", "softplus", "seqs", "rows", "channels", "groups", "states")] + [
        ("starts", _P)] + [(n, Rows) for n in ("u", "delta", "z", "out", "B", "C")] + [
        (n, _P) for n in ("A", "D", "delta_bias", "init_state", "final_state",
                          "chunk_states")] + [
        (n, Rows) for n in ("dout", "du", "ddelta", "dz", "dB", "dC")] + [
        (n, _P) for n in ("dA", "dD", "ddelta_bias", "d_final_state", "d_init_state")]


_seq = None


def _lib() -> ctypes.CDLL:
    global _seq
    if _seq is not None:
        return _seq
    L = lib()
    S, I, F = ctypes.c_size_t, ctypes.c_int, ctypes.c_float
    for name in SEQ_EXPORTS:
        f = getattr(L, name)
        f.restype = S if name.endswith("_bytes") or name.endswith("_states") else I
    L.canon_embedding.argtypes = [I, _P, S, S, S, _P, I, S, F, _P, S, _P]
    L.canon_embedding_grad_workspace_bytes.argtypes = [S, S, S]
    L.canon_embedding_grad.argtypes = [I, _P, S, _P, I, S, S, S, F, _I64, I, I, _P, S, _P, S, _P]
    L.canon_causal_conv.argtypes = [_P, _P]
    L.canon_causal_conv_grad_workspace_bytes.argtypes = [S, S, I, S, S]
    L.canon_causal_conv_grad.argtypes = [_P, _P, S, _P]
    L.canon_causal_conv_step.argtypes = [_P, _P]
    L.canon_selective_scan_states.argtypes = [S, S, I, S, S]
    L.canon_selective_scan_workspace_bytes.argtypes = [S, S, I, S, S]
    L.canon_selective_scan.argtypes = [_P, _P, S, _P]
    L.canon_selective_scan_grad_workspace_bytes.argtypes = [S, S, I, S, S, S]
    L.canon_selective_scan_grad.argtypes = [_P, _P, S, _P]
    L.canon_selective_scan_step.argtypes = [_P, _P]
    if L.canon_seq_version() != SEQ_VERSION:
        raise CanonError("libcanon sequence operators: version mismatch")
    _seq = L
    return L


# ------------------------------------------------------------------- arguments
def _dtype(t: torch.Tensor, what: str) -> int:
    d = DTYPES.get(t.dtype)
    if d is None:
        raise TypeError(f"{what} takes float32, bfloat16 or float16, not {t.dtype}")
    return d


def _same(what: str, device: torch.device, *ts: Optional[torch.Tensor]) -> None:
    """Every tensor on `device`, a GPU (there is no CPU path)."""
    if device.type != "cuda":
        raise ValueError("tensors must live on the GPU (no CPU path)")
    for t in ts:
        if t is not None and t.device != device:
            raise ValueError(f"{what}: tensors are on {device} and {t.device}")


class _On:
    """The device of a call, made current if it is not, and its stream."""
    __slots__ = ("device", "guard")

    def __init__(self, device: torch.device):
        self.device = device
        self.guard = None

    def __enter__(self) -> int:
        if self.device.index != torch.cuda.current_device():
            self.guard = torch.cuda.device(self.device)
            self.guard.__enter__()
        return torch.cuda.current_stream(self.device).cuda_stream

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)
        return False


def _shape(what: str, name: str, t: torch.Tensor, shape, dtype=None) -> None:
    if t.shape != tuple(shape) or (dtype is not None and t.dtype != dtype):
        want = f" {dtype}" if dtype is not None else ""
        raise ValueError(f"{what}: {name} must be{want} of shape {tuple(shape)}, "
                         f"not {t.dtype} {tuple(t.shape)}")


def _flat(what: str, name: str, t: Optional[torch.Tensor], shape, dtype) -> Optional[int]:
    """Pointer of a contiguous tensor of that shape and type (None if absent)."""
    if t is None:
        return None
    _shape(what, name, t, shape, dtype)
    if not t.is_contiguous():
        raise ValueError(f"{what}: {name} must be contiguous")
    return t.data_ptr()


def _rows(what: str, name: str, t: torch.Tensor, shape, dtype, lead: int) -> Rows:
    """canon_rows_t of an activation whose first `lead` dimensions are rows
    (1), or sequences and rows (2); the others are its columns, contiguous.
    Strides of dimensions of one element are never used and passed as 0."""
    _shape(what, name, t, shape, dtype)
    st = t.stride()
    run = 1
    for i in range(t.dim() - 1, lead - 1, -1):
        if shape[i] != 1 and st[i] != run and t.numel():
            raise ValueError(f"{what}: the columns of {name} must be contiguous")
        run *= shape[i]
    return Rows(t.data_ptr(), st[0] if lead == 2 and shape[0] > 1 else 0,
                st[lead - 1] if shape[lead - 1] > 1 else 0)


_NONE = Rows(None, 0, 0)


def _sequences(what: str, x: torch.Tensor, starts: Optional[torch.Tensor]):
    """(sequences, rows, pointer of starts, leading dimensions)"""
    if starts is None:
        if x.dim() != 3:
            raise ValueError(f"{what} takes [sequences, rows, channels], or packed rows with "
                             "starts")
        return x.shape[0], x.shape[1], None, 2
    if x.dim() != 2:
        raise ValueError(f"{what} with starts takes [rows, channels]")
    if starts.dtype != torch.int32 or starts.dim() != 1 or starts.numel() < 1 \
            or not starts.is_contiguous():
        raise ValueError(f"{what}: starts must be a contiguous 1-d int32 tensor of at least 1")
    return starts.numel() - 1, x.shape[0], starts.data_ptr(), 1


def _workspace(nbytes: int, device: torch.device, ws: Optional[torch.Tensor]):
    if ws is not None and ws.numel() >= nbytes:
        if ws.dtype != torch.uint8 or not ws.is_contiguous() or ws.device != device:
            raise ValueError(f"ws must be a contiguous uint8 tensor on {device}")
        return ws
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


# ------------------------------------------------------------------- embedding
def _matrix(what: str, name: str, t: torch.Tensor):
    if t.dim() != 2 or (t.shape[1] > 1 and t.numel() and t.stride(1) != 1):
        raise ValueError(f"{what}: {name} must be 2-d with unit column stride")
    rows, cols = t.shape
    ld = t.stride(0) if rows > 1 else cols
    if ld < cols:
        raise ValueError(f"{what}: rows of {name} overlap")
    return rows, cols, ld


def _ids(what: str, ids: torch.Tensor):
    if ids.dtype not in (torch.int64, torch.int32) or not ids.is_contiguous():
        raise ValueError(f"{what}: ids must be a contiguous int64 or int32 tensor")
    return ids.data_ptr(), ids.element_size(), ids.numel()


def embedding(weight: torch.Tensor, ids: torch.Tensor, scale: float = 1.0,
              out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """scale * weight[ids], of shape ids.shape + (width,); a zero row for an id
    outside the table."""
    what = "embedding"
    _same(what, weight.device, ids, out)
    d = _dtype(weight, what)
    rows, width, ld = _matrix(what, "weight", weight)
    p, nb, tokens = _ids(what, ids)
    if out is None:
        out = torch.empty(ids.shape + (width,), dtype=weight.dtype, device=weight.device)
    _shape(what, "out", out, ids.shape + (width,), weight.dtype)
    if out.dim() != 2:
        if not out.is_contiguous():
            raise ValueError(f"{what}: out must be contiguous unless it is 2-d")
        ld_out = width
    else:
        ld_out = _matrix(what, "out", out)[2]
    with _On(weight.device) as stream:
        st = _lib().canon_embedding(d, weight.data_ptr(), ld, rows, width, p, nb, tokens, scale,
                                    out.data_ptr(), ld_out, stream)
    _check(st, what)
    return out


def embedding_grad_workspace_bytes(tokens: int, rows: int, width: int) -> int:
    return _lib().canon_embedding_grad_workspace_bytes(tokens, rows, width)


def embedding_grad(dout: torch.Tensor, ids: torch.Tensor, rows: int, scale: float = 1.0,
                   padding_id: Optional[int] = None, out: Optional[torch.Tensor] = None,
                   accumulate: bool = False, dtype: Optional[torch.dtype] = None,
                   ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of embedding's table (`rows` rows): row v is scale times the
    pairwise-tree sum (canon.h) of the rows of dout whose id is v, in token
    order.  Ids outside the table and padding_id add nothing.  dtype (or
    out's): dout's type or float32.  accumulate: added to out."""
    what = "embedding_grad"
    _same(what, dout.device, ids, out, ws)
    d = _dtype(dout, what)
    p, nb, tokens = _ids(what, ids)
    width = dout.shape[-1] if dout.dim() else 0
    if dout.dim() < 1 or dout.shape[:-1] != ids.shape:
        raise ValueError(f"{what}: dout must have one row per id")
    if dout.dim() != 2:
        if not dout.is_contiguous():
            raise ValueError(f"{what}: dout must be contiguous unless it is 2-d")
        ld = width
    else:
        ld = _matrix(what, "dout", dout)[2]
    if padding_id is not None and padding_id < 0:
        raise ValueError(f"{what}: padding_id must not be negative (such ids add nothing)")
    if out is None:
        if accumulate:
            raise ValueError(f"{what}: accumulate needs out")
        out = torch.empty((rows, width), dtype=dtype or dout.dtype, device=dout.device)
    _shape(what, "out", out, (rows, width), dtype)
    if out.dtype not in (dout.dtype, torch.float32):
        raise TypeError(f"{what}: the gradient must be {dout.dtype} or float32, not {out.dtype}")
    ld_out = _matrix(what, "out", out)[2]
    L = _lib()
    n = L.canon_embedding_grad_workspace_bytes(tokens, rows, width)
    with _On(dout.device) as stream:
        w = _workspace(n, dout.device, ws)
        st = L.canon_embedding_grad(d, dout.data_ptr(), ld, p, nb, tokens, rows, width, scale,
                                    -1 if padding_id is None else padding_id, int(accumulate),
                                    DTYPES[out.dtype], out.data_ptr(), ld_out, w.data_ptr(),
                                    w.numel(), stream)
    _check(st, what)
    return out


# ---------------------------------------------------------- causal convolution
class CausalConvGrads(NamedTuple):
    dx: torch.Tensor
    dweight: torch.Tensor
    dbias: Optional[torch.Tensor]
    dinit_state: Optional[torch.Tensor]


def _activation(what: str, a) -> int:
    if a not in (None, "silu"):
        raise ValueError(f"{what}: activation must be None or \"silu\", not {a!r}")
    return int(a == "silu")


def _conv(what, x, weight, bias, activation, seqs, rows, starts, lead) -> Conv:
    c = Conv()
    c.dtype = _dtype(x, what)
    channels = x.shape[-1]
    if weight.dim() != 2 or weight.shape[0] != channels:
        raise ValueError(f"{what}: weight must be [{channels}, taps]")
    c.taps = weight.shape[1]
    c.silu = _activation(what, activation)
    if weight.dtype not in (x.dtype, torch.float32):
        raise TypeError(f"{what}: weight must be {x.dtype} or float32, not {weight.dtype}")
    c.param_dtype = DTYPES[weight.dtype]
    c.seqs, c.rows, c.channels, c.starts = seqs, rows, channels, starts
    c.x = _rows(what, "x", x, x.shape, x.dtype, lead)
    c.weight = _flat(what, "weight", weight, weight.shape, weight.dtype)
    c.bias = _flat(what, "bias", bias, (channels,), weight.dtype)
    return c


def causal_conv(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                activation: Optional[str] = None, starts: Optional[torch.Tensor] = None,
                init_state: Optional[torch.Tensor] = None,
                final_state: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Depthwise causal convolution over the rows of each sequence, weight
    [channels, taps] (float32 or x's type, as bias), activation None or "silu".
    init_state, final_state: [sequences, taps - 1, channels] of x's type, the
    rows before the first and the last rows seen (final_state is written, and
    may be init_state)."""
    what = "causal_conv"
    _same(what, x.device, weight, bias, starts, init_state, final_state, out)
    seqs, rows, sp, lead = _sequences(what, x, starts)
    c = _conv(what, x, weight, bias, activation, seqs, rows, sp, lead)
    state = (seqs, c.taps - 1, x.shape[-1])
    c.init_state = _flat(what, "init_state", init_state, state, x.dtype)
    c.final_state = _flat(what, "final_state", final_state, state, x.dtype)
    with _On(x.device) as stream:
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        c.out = _rows(what, "out", out, x.shape, x.dtype, lead)
        _check(_lib().canon_causal_conv(ctypes.byref(c), stream), what)
    return out


def causal_conv_grad_workspace_bytes(seqs: int, rows: int, packed: bool, channels: int,
                                     taps: int) -> int:
    return _lib().canon_causal_conv_grad_workspace_bytes(seqs, rows, int(packed), channels, taps)


def causal_conv_grad(dout: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                     bias: Optional[torch.Tensor] = None, activation: Optional[str] = None,
                     starts: Optional[torch.Tensor] = None,
                     init_state: Optional[torch.Tensor] = None,
                     d_final_state: Optional[torch.Tensor] = None,
                     dx: Optional[torch.Tensor] = None,
                     ws: Optional[torch.Tensor] = None) -> CausalConvGrads:
    """Gradients of causal_conv's inputs; dweight and dbias are float32,
    dinit_state (with init_state) has x's type.  Rows of dx that belong to no
    sequence are left as they are."""
    what = "causal_conv_grad"
    _same(what, x.device, dout, weight, bias, starts, init_state, d_final_state, dx, ws)
    seqs, rows, sp, lead = _sequences(what, x, starts)
    c = _conv(what, x, weight, bias, activation, seqs, rows, sp, lead)
    channels = x.shape[-1]
    state = (seqs, c.taps - 1, channels)
    c.init_state = _flat(what, "init_state", init_state, state, x.dtype)
    c.d_final_state = _flat(what, "d_final_state", d_final_state, state, x.dtype)
    c.dout = _rows(what, "dout", dout, x.shape, x.dtype, lead)
    L = _lib()
    n = L.canon_causal_conv_grad_workspace_bytes(seqs, rows, int(sp is not None), channels, c.taps)
    with _On(x.device) as stream:
        if dx is None:
            dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        dw = torch.empty(weight.shape, dtype=torch.float32, device=x.device)
        db = None if bias is None else torch.empty(channels, dtype=torch.float32, device=x.device)
        di = None if init_state is None else torch.empty_like(init_state)
        w = _workspace(n, x.device, ws)
        c.dx = _rows(what, "dx", dx, x.shape, x.dtype, lead)
        c.dweight = dw.data_ptr()
        c.dbias = None if db is None else db.data_ptr()
        c.d_init_state = None if di is None else di.data_ptr()
        _check(L.canon_causal_conv_grad(ctypes.byref(c), w.data_ptr(), w.numel(), stream), what)
    return CausalConvGrads(dx, dw, db, di)


def causal_conv_step(x: torch.Tensor, state: torch.Tensor, weight: torch.Tensor,
                     bias: Optional[torch.Tensor] = None, activation: Optional[str] = None,
                     out_state: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """causal_conv for one row of each sequence: x [sequences, channels].  The
    state [sequences, taps - 1, channels] is updated in place, or, with
    out_state, read and written there."""
    what = "causal_conv_step"
    _same(what, x.device, weight, bias, state, out_state, out)
    if x.dim() != 2:
        raise ValueError(f"{what} takes [sequences, channels]")
    c = _conv(what, x, weight, bias, activation, x.shape[0], 1, None, 1)
    c.x = Rows(c.x.p, c.x.row, 0)
    shape = (x.shape[0], c.taps - 1, x.shape[1])
    c.init_state = _flat(what, "state", state, shape, x.dtype)
    c.final_state = c.init_state if out_state is None else \
        _flat(what, "out_state", out_state, shape, x.dtype)
    with _On(x.device) as stream:
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        o = _rows(what, "out", out, x.shape, x.dtype, 1)
        c.out = Rows(o.p, o.row, 0)
        _check(_lib().canon_causal_conv_step(ctypes.byref(c), stream), what)
    return out


# --------------------------------------------------------------- selective scan
class SelectiveScanGrads(NamedTuple):
    du: torch.Tensor
    ddelta: torch.Tensor
    dA: torch.Tensor
    dB: torch.Tensor
    dC: torch.Tensor
    dD: Optional[torch.Tensor]
    dz: Optional[torch.Tensor]
    ddelta_bias: Optional[torch.Tensor]
    dinit_state: Optional[torch.Tensor]


def _scan(what, u, delta, A, B, C, D, z, delta_bias, softplus, seqs, rows, starts, lead) -> Scan:
    c = Scan()
    c.dtype = _dtype(u, what)
    channels = u.shape[-1]
    if A.dim() != 2 or A.shape[0] != channels:
        raise ValueError(f"{what}: A must be [{channels}, states]")
    states = A.shape[1]
    groups = B.shape[-2] if B.dim() == u.dim() + 1 else 1
    bc = u.shape[:-1] + ((groups, states) if B.dim() == u.dim() + 1 else (states,))
    if groups < 1 or channels % groups:
        raise ValueError(f"{what}: {channels} channels do not divide into {groups} groups")
    c.softplus = int(bool(softplus))
    c.seqs, c.rows, c.channels, c.groups, c.states = seqs, rows, channels, groups, states
    c.starts = starts
    c.u = _rows(what, "u", u, u.shape, u.dtype, lead)
    c.delta = _rows(what, "delta", delta, u.shape, u.dtype, lead)
    c.B = _rows(what, "B", B, bc, u.dtype, lead)
    c.C = _rows(what, "C", C, bc, u.dtype, lead)
    if z is not None:
        c.z = _rows(what, "z", z, u.shape, u.dtype, lead)
    f32 = torch.float32
    c.A = _flat(what, "A", A, A.shape, f32)
    c.D = _flat(what, "D", D, (channels,), f32)
    c.delta_bias = _flat(what, "delta_bias", delta_bias, (channels,), f32)
    return c


def selective_scan_workspace_bytes(seqs: int, rows: int, packed: bool, channels: int,
                                   states: int) -> int:
    return _lib().canon_selective_scan_workspace_bytes(seqs, rows, int(packed), channels, states)


def selective_scan_grad_workspace_bytes(seqs: int, rows: int, packed: bool, channels: int,
                                        groups: int, states: int) -> int:
    return _lib().canon_selective_scan_grad_workspace_bytes(seqs, rows, int(packed), channels,
                                                            groups, states)


def selective_scan_states(u: torch.Tensor, states: int,
                          starts: Optional[torch.Tensor] = None) -> torch.Tensor:
    """An uninitialised buffer for selective_scan's `states` argument: what the
    forward pass of u saves for the backward pass (4 bytes per element of u and
    16 states)."""
    seqs, rows, sp, _ = _sequences("selective_scan_states", u, starts)
    n = _lib().canon_selective_scan_states(seqs, rows, int(sp is not None), u.shape[-1], states)
    return torch.empty(n, dtype=torch.float32, device=u.device)


def selective_scan(u: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                   C: torch.Tensor, D: Optional[torch.Tensor] = None,
                   z: Optional[torch.Tensor] = None, delta_bias: Optional[torch.Tensor] = None,
                   delta_softplus: bool = False, starts: Optional[torch.Tensor] = None,
                   init_state: Optional[torch.Tensor] = None,
                   final_state: Optional[torch.Tensor] = None,
                   states: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The selective state space scan of each sequence.

    u, delta, z: activations of the same shape; A [channels, states]; B, C with
    u's leading dimensions and [states] or [groups, states] columns; D,
    delta_bias [channels].  init_state, final_state [sequences, channels,
    states]: the state before the first row and after the last (written, and
    may be init_state).  states: a buffer of selective_scan_states for the
    backward pass."""
    what = "selective_scan"
    _same(what, u.device, delta, A, B, C, D, z, delta_bias, starts, init_state, final_state,
          states, out, ws)
    seqs, rows, sp, lead = _sequences(what, u, starts)
    c = _scan(what, u, delta, A, B, C, D, z, delta_bias, delta_softplus, seqs, rows, sp, lead)
    shape = (seqs, c.channels, c.states)
    c.init_state = _flat(what, "init_state", init_state, shape, torch.float32)
    c.final_state = _flat(what, "final_state", final_state, shape, torch.float32)
    L = _lib()
    if states is not None:
        n = L.canon_selective_scan_states(seqs, rows, int(sp is not None), c.channels, c.states)
        c.chunk_states = _flat(what, "states", states, (n,), torch.float32)
    n = L.canon_selective_scan_workspace_bytes(seqs, rows, int(sp is not None), c.channels,
                                               c.states)
    with _On(u.device) as stream:
        if out is None:
            out = torch.empty(u.shape, dtype=u.dtype, device=u.device)
        c.out = _rows(what, "out", out, u.shape, u.dtype, lead)
        w = _workspace(n, u.device, ws)
        _check(L.canon_selective_scan(ctypes.byref(c), w.data_ptr(), w.numel(), stream), what)
    return out


def selective_scan_grad(dout: torch.Tensor, u: torch.Tensor, delta: torch.Tensor,
                        A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                        states: torch.Tensor, D: Optional[torch.Tensor] = None,
                        z: Optional[torch.Tensor] = None,
                        delta_bias: Optional[torch.Tensor] = None, delta_softplus: bool = False,
                        starts: Optional[torch.Tensor] = None,
                        d_final_state: Optional[torch.Tensor] = None,
                        ws: Optional[torch.Tensor] = None) -> SelectiveScanGrads:
    """Gradients of selective_scan's inputs, given the `states` that its call
    with these inputs wrote, and the gradients of its output and (optionally)
    final state.  Activations' gradients have their type, the others are
    float32; rows that belong to no sequence have undefined gradients."""
    what = "selective_scan_grad"
    _same(what, u.device, dout, delta, A, B, C, D, z, delta_bias, starts, states, d_final_state,
          ws)
    seqs, rows, sp, lead = _sequences(what, u, starts)
    c = _scan(what, u, delta, A, B, C, D, z, delta_bias, delta_softplus, seqs, rows, sp, lead)
    shape = (seqs, c.channels, c.states)
    f32, device = torch.float32, u.device
    c.dout = _rows(what, "dout", dout, u.shape, u.dtype, lead)
    c.d_final_state = _flat(what, "d_final_state", d_final_state, shape, f32)
    L = _lib()
    n = L.canon_selective_scan_states(seqs, rows, int(sp is not None), c.channels, c.states)
    c.chunk_states = _flat(what, "states", states, (n,), f32)
    n = L.canon_selective_scan_grad_workspace_bytes(seqs, rows, int(sp is not None), c.channels,
                                                    c.groups, c.states)
    with _On(device) as stream:
        w = _workspace(n, device, ws)
        g = SelectiveScanGrads(
            du=torch.empty(u.shape, dtype=u.dtype, device=device),
            ddelta=torch.empty(u.shape, dtype=u.dtype, device=device),
            dA=torch.empty(A.shape, dtype=f32, device=device),
            dB=torch.empty(B.shape, dtype=u.dtype, device=device),
            dC=torch.empty(C.shape, dtype=u.dtype, device=device),
            dD=None if D is None else torch.empty(c.channels, dtype=f32, device=device),
            dz=None if z is None else torch.empty(u.shape, dtype=u.dtype, device=device),
            ddelta_bias=None if delta_bias is None else
            torch.empty(c.channels, dtype=f32, device=device),
            dinit_state=torch.empty(shape, dtype=f32, device=device))
        c.du = _rows(what, "du", g.du, u.shape, u.dtype, lead)
        c.ddelta = _rows(what, "ddelta", g.ddelta, u.shape, u.dtype, lead)
        c.dB = _rows(what, "dB", g.dB, B.shape, u.dtype, lead)
        c.dC = _rows(what, "dC", g.dC, C.shape, u.dtype, lead)
        if z is not None:
            c.dz = _rows(what, "dz", g.dz, u.shape, u.dtype, lead)
        c.dA = g.dA.data_ptr()
        c.dD = None if D is None else g.dD.data_ptr()
        c.ddelta_bias = None if delta_bias is None else g.ddelta_bias.data_ptr()
        c.d_init_state = g.dinit_state.data_ptr()
        _check(L.canon_selective_scan_grad(ctypes.byref(c), w.data_ptr(), w.numel(), stream), what)
    return g


def selective_scan_step(state: torch.Tensor, u: torch.Tensor, delta: torch.Tensor,
                        A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                        D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                        delta_bias: Optional[torch.Tensor] = None, delta_softplus: bool = False,
                        out_state: Optional[torch.Tensor] = None,
                        out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """selective_scan for one row of each sequence: u, delta, z [sequences,
    channels]; B, C [sequences, states] or [sequences, groups, states].  The
    state [sequences, channels, states] is updated in place, or, with
    out_state, read and written there."""
    what = "selective_scan_step"
    _same(what, u.device, state, delta, A, B, C, D, z, delta_bias, out_state, out)
    if u.dim() != 2:
        raise ValueError(f"{what} takes [sequences, channels]")
    c = _scan(what, u, delta, A, B, C, D, z, delta_bias, delta_softplus, u.shape[0], 1, None, 1)
    for name in ("u", "delta", "z", "B", "C"):  # one row per sequence
        r = getattr(c, name)
        setattr(c, name, Rows(r.p, r.row, 0))
    shape = (u.shape[0], c.channels, c.states)
    c.init_state = _flat(what, "state", state, shape, torch.float32)
    c.final_state = c.init_state if out_state is None else \
        _flat(what, "out_state", out_state, shape, torch.float32)
    with _On(u.device) as stream:
        if out is None:
            out = torch.empty(u.shape, dtype=u.dtype, device=u.device)
        o = _rows(what, "out", out, u.shape, u.dtype, 1)
        c.out = Rows(o.p, o.row, 0)
        _check(_lib().canon_selective_scan_step(ctypes.byref(c), stream), what)
    return out
