"""Operators of sequence models: embedding, causal convolution, selective scan.

Argument marshalling only, as in the package itself; the C ABI is declared in
``include/canon_seq.h``, which states what each operator computes.

Shapes.  Activations (float32, bfloat16 or float16, one type per call) are
``[sequences, rows, columns]``, or with ``starts`` (int32, sequences + 1
ascending row offsets, on the GPU) ``[rows, columns]`` with the sequences
packed one after the other; rows outside them are left as they are.  Columns
have unit stride, rows and sequences any.  Parameters, their gradients and scan
states are float32 and contiguous, the convolution's states contiguous and of the
activations' type.

Calls run on the current stream of the tensors' device.  ``ws`` is a
caller-owned uint8 workspace of ``*_workspace_bytes(...)`` bytes; without it,
or if it is too small, the call allocates its own.
"""
from __future__ import annotations

import ctypes
import struct
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

# canon_conv_t and canon_selective_scan_t: fields of 8 bytes, pointers included
# (0: NULL), a canon_rows_t being three of them.  Packed in one go: a call's time
# is mostly the host's for small sizes, and a ctypes structure filled field by
# field takes three microseconds more.
CONV = struct.Struct("=28q")
SCAN = struct.Struct("=55q")
_NONE = (0, 0, 0)


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


def _call(what: str, device: torch.device, fn, *args) -> None:
    """fn(*args, stream) on the device's current stream, the device made
    current if it is not."""
    index = device.index
    stream = torch._C._cuda_getCurrentRawStream(index)
    if index == torch._C._cuda_getDevice():
        st = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            st = fn(*args, stream)
    if st:
        _check(st, what)


def _wrong(what: str, name: str, t: torch.Tensor, shape, dtype) -> ValueError:
    return ValueError(f"{what}: {name} must be {dtype} of shape {tuple(shape)}, "
                      f"not {t.dtype} {tuple(t.shape)}")


def _flat(what: str, name: str, t: Optional[torch.Tensor], shape, dtype) -> int:
    """Pointer of a contiguous tensor of that shape and type (0 if absent)."""
    if t is None:
        return 0
    if t.shape != shape or t.dtype != dtype:
        raise _wrong(what, name, t, shape, dtype)
    if not t.is_contiguous():
        raise ValueError(f"{what}: {name} must be contiguous")
    return t.data_ptr()


def _rows(what: str, name: str, t: torch.Tensor, shape, dtype, lead: int):
    """canon_rows_t of an activation whose first `lead` dimensions are rows
    (1), or sequences and rows (2); the one or two others are its columns,
    contiguous.  Strides of dimensions of one element are never used and passed
    as 0."""
    if t.shape != shape or t.dtype != dtype:
        raise _wrong(what, name, t, shape, dtype)
    st = t.stride()
    cols = shape[-1]
    if ((st[-1] != 1 and cols != 1)
            or (len(st) > lead + 1 and st[-2] != cols and shape[-2] != 1)) and t.numel():
        raise ValueError(f"{what}: the columns of {name} must be contiguous")
    row = st[lead - 1] if shape[lead - 1] > 1 else 0
    if lead == 1:
        return t.data_ptr(), 0, row
    return t.data_ptr(), st[0] if shape[0] > 1 else 0, row


def _step_rows(what: str, name: str, t: torch.Tensor, shape, dtype):
    """canon_rows_t of one row per sequence."""
    p, _, row = _rows(what, name, t, shape, dtype, 1)
    return p, row, 0


def _sequences(what: str, x: torch.Tensor, starts: Optional[torch.Tensor]):
    """(sequences, rows, pointer of starts, leading dimensions)"""
    if starts is None:
        if x.dim() != 3:
            raise ValueError(f"{what} takes [sequences, rows, channels], or packed rows with "
                             "starts")
        return x.shape[0], x.shape[1], 0, 2
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
    shape = ids.shape + (width,)
    if out is None:
        out = weight.new_empty(shape)
        ld_out = width
    elif out.shape != shape or out.dtype != weight.dtype:
        raise _wrong(what, "out", out, shape, weight.dtype)
    elif out.dim() == 2:
        ld_out = _matrix(what, "out", out)[2]
    elif out.is_contiguous():
        ld_out = width
    else:
        raise ValueError(f"{what}: out must be contiguous unless it is 2-d")
    _call(what, weight.device, _lib().canon_embedding, d, weight.data_ptr(), ld, rows, width, p,
          nb, tokens, scale, out.data_ptr(), ld_out)
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
    elif out.shape != (rows, width) or (dtype is not None and out.dtype != dtype):
        raise _wrong(what, "out", out, (rows, width), dtype or out.dtype)
    if out.dtype != dout.dtype and out.dtype != torch.float32:
        raise TypeError(f"{what}: the gradient must be {dout.dtype} or float32, not {out.dtype}")
    ld_out = _matrix(what, "out", out)[2]
    L = _lib()
    w = _workspace(L.canon_embedding_grad_workspace_bytes(tokens, rows, width), dout.device, ws)
    _call(what, dout.device, L.canon_embedding_grad, d, dout.data_ptr(), ld, p, nb, tokens, rows,
          width, scale, -1 if padding_id is None else padding_id, int(accumulate),
          DTYPES[out.dtype], out.data_ptr(), ld_out, w.data_ptr(), w.numel())
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


def _conv(what, x, weight, bias, activation):
    """(dtype, taps, silu, param_dtype), channels, (weight, bias)"""
    d = _dtype(x, what)
    channels = x.shape[-1]
    if weight.dim() != 2 or weight.shape[0] != channels:
        raise ValueError(f"{what}: weight must be [{channels}, taps]")
    if weight.dtype != x.dtype and weight.dtype != torch.float32:
        raise TypeError(f"{what}: weight must be {x.dtype} or float32, not {weight.dtype}")
    head = (d, weight.shape[1], _activation(what, activation), DTYPES[weight.dtype])
    return head, channels, (_flat(what, "weight", weight, weight.shape, weight.dtype),
                            _flat(what, "bias", bias, (channels,), weight.dtype))


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
    head, channels, params = _conv(what, x, weight, bias, activation)
    state = (seqs, head[1] - 1, channels)
    if out is None:
        out = x.new_empty(x.shape)
    c = CONV.pack(*head, seqs, rows, channels, sp, *_rows(what, "x", x, x.shape, x.dtype, lead),
                  *_rows(what, "out", out, x.shape, x.dtype, lead), *params,
                  _flat(what, "init_state", init_state, state, x.dtype),
                  _flat(what, "final_state", final_state, state, x.dtype),
                  *_NONE, *_NONE, 0, 0, 0, 0)
    _call(what, x.device, _lib().canon_causal_conv, c)
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
    head, channels, params = _conv(what, x, weight, bias, activation)
    state = (seqs, head[1] - 1, channels)
    device = x.device
    if dx is None:
        dx = x.new_empty(x.shape)
    dw = torch.empty(weight.shape, dtype=torch.float32, device=device)
    db = None if bias is None else torch.empty(channels, dtype=torch.float32, device=device)
    di = None if init_state is None else torch.empty_like(init_state)
    c = CONV.pack(*head, seqs, rows, channels, sp, *_rows(what, "x", x, x.shape, x.dtype, lead),
                  *_NONE, *params, _flat(what, "init_state", init_state, state, x.dtype), 0,
                  *_rows(what, "dout", dout, x.shape, x.dtype, lead),
                  *_rows(what, "dx", dx, x.shape, x.dtype, lead), dw.data_ptr(),
                  0 if db is None else db.data_ptr(),
                  _flat(what, "d_final_state", d_final_state, state, x.dtype),
                  0 if di is None else di.data_ptr())
    L = _lib()
    w = _workspace(L.canon_causal_conv_grad_workspace_bytes(seqs, rows, int(lead == 1), channels,
                                                            head[1]), device, ws)
    _call(what, device, L.canon_causal_conv_grad, c, w.data_ptr(), w.numel())
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
    head, channels, params = _conv(what, x, weight, bias, activation)
    shape = (x.shape[0], head[1] - 1, channels)
    old = _flat(what, "state", state, shape, x.dtype)
    if out is None:
        out = x.new_empty(x.shape)
    c = CONV.pack(*head, x.shape[0], 1, channels, 0, *_step_rows(what, "x", x, x.shape, x.dtype),
                  *_step_rows(what, "out", out, x.shape, x.dtype), *params, old,
                  old if out_state is None else _flat(what, "out_state", out_state, shape, x.dtype),
                  *_NONE, *_NONE, 0, 0, 0, 0)
    _call(what, x.device, _lib().canon_causal_conv_step, c)
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


def _scan(what, u, A, B, D, delta_bias, softplus):
    """(dtype, softplus), (channels, groups, states), shape of B and C, (A, D,
    delta_bias)"""
    d = _dtype(u, what)
    channels = u.shape[-1]
    if A.dim() != 2 or A.shape[0] != channels:
        raise ValueError(f"{what}: A must be [{channels}, states]")
    states = A.shape[1]
    if B.dim() == u.dim() + 1:
        groups = B.shape[-2]
        bc = u.shape[:-1] + (groups, states)
    else:
        groups = 1
        bc = u.shape[:-1] + (states,)
    if groups < 1 or channels % groups:
        raise ValueError(f"{what}: {channels} channels do not divide into {groups} groups")
    f32 = torch.float32
    return (d, int(bool(softplus))), (channels, groups, states), bc, (
        _flat(what, "A", A, A.shape, f32), _flat(what, "D", D, (channels,), f32),
        _flat(what, "delta_bias", delta_bias, (channels,), f32))


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
    seqs, rows, _, lead = _sequences("selective_scan_states", u, starts)
    n = _lib().canon_selective_scan_states(seqs, rows, int(lead == 1), u.shape[-1], states)
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
    head, sizes, bc, params = _scan(what, u, A, B, D, delta_bias, delta_softplus)
    channels, _, n = sizes
    shape, f32, dtype, packed = (seqs, channels, n), torch.float32, u.dtype, int(lead == 1)
    L = _lib()
    kept = 0
    if states is not None:
        size = L.canon_selective_scan_states(seqs, rows, packed, channels, n)
        kept = _flat(what, "states", states, (size,), f32)
    if out is None:
        out = u.new_empty(u.shape)
    c = SCAN.pack(*head, seqs, rows, *sizes, sp, *_rows(what, "u", u, u.shape, dtype, lead),
                  *_rows(what, "delta", delta, u.shape, dtype, lead),
                  *(_NONE if z is None else _rows(what, "z", z, u.shape, dtype, lead)),
                  *_rows(what, "out", out, u.shape, dtype, lead),
                  *_rows(what, "B", B, bc, dtype, lead), *_rows(what, "C", C, bc, dtype, lead),
                  *params, _flat(what, "init_state", init_state, shape, f32),
                  _flat(what, "final_state", final_state, shape, f32), kept, *_NONE, *_NONE,
                  *_NONE, *_NONE, *_NONE, *_NONE, 0, 0, 0, 0, 0)
    w = _workspace(L.canon_selective_scan_workspace_bytes(seqs, rows, packed, channels, n),
                   u.device, ws)
    _call(what, u.device, L.canon_selective_scan, c, w.data_ptr(), w.numel())
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
    head, sizes, bc, params = _scan(what, u, A, B, D, delta_bias, delta_softplus)
    channels, groups, n = sizes
    shape, f32, packed = (seqs, channels, n), torch.float32, int(lead == 1)
    device, dtype = u.device, u.dtype
    L = _lib()
    size = L.canon_selective_scan_states(seqs, rows, packed, channels, n)
    g = SelectiveScanGrads(
        du=u.new_empty(u.shape), ddelta=u.new_empty(u.shape), dA=A.new_empty(A.shape),
        dB=u.new_empty(bc), dC=u.new_empty(bc), dD=None if D is None else D.new_empty(channels),
        dz=None if z is None else u.new_empty(u.shape),
        ddelta_bias=None if delta_bias is None else delta_bias.new_empty(channels),
        dinit_state=A.new_empty(shape))
    c = SCAN.pack(*head, seqs, rows, *sizes, sp, *_rows(what, "u", u, u.shape, dtype, lead),
                  *_rows(what, "delta", delta, u.shape, dtype, lead),
                  *(_NONE if z is None else _rows(what, "z", z, u.shape, dtype, lead)), *_NONE,
                  *_rows(what, "B", B, bc, dtype, lead), *_rows(what, "C", C, bc, dtype, lead),
                  *params, 0, 0, _flat(what, "states", states, (size,), f32),
                  *_rows(what, "dout", dout, u.shape, dtype, lead),
                  *_rows(what, "du", g.du, u.shape, dtype, lead),
                  *_rows(what, "ddelta", g.ddelta, u.shape, dtype, lead),
                  *(_NONE if z is None else _rows(what, "dz", g.dz, u.shape, dtype, lead)),
                  *_rows(what, "dB", g.dB, bc, dtype, lead),
                  *_rows(what, "dC", g.dC, bc, dtype, lead), g.dA.data_ptr(),
                  0 if D is None else g.dD.data_ptr(),
                  0 if delta_bias is None else g.ddelta_bias.data_ptr(),
                  _flat(what, "d_final_state", d_final_state, shape, f32),
                  g.dinit_state.data_ptr())
    w = _workspace(L.canon_selective_scan_grad_workspace_bytes(seqs, rows, packed, channels,
                                                               groups, n), device, ws)
    _call(what, device, L.canon_selective_scan_grad, c, w.data_ptr(), w.numel())
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
    head, sizes, bc, params = _scan(what, u, A, B, D, delta_bias, delta_softplus)
    seqs, dtype, f32 = u.shape[0], u.dtype, torch.float32
    shape = (seqs, sizes[0], sizes[2])
    old = _flat(what, "state", state, shape, f32)
    if out is None:
        out = u.new_empty(u.shape)
    c = SCAN.pack(*head, seqs, 1, *sizes, 0, *_step_rows(what, "u", u, u.shape, dtype),
                  *_step_rows(what, "delta", delta, u.shape, dtype),
                  *(_NONE if z is None else _step_rows(what, "z", z, u.shape, dtype)),
                  *_step_rows(what, "out", out, u.shape, dtype),
                  *_step_rows(what, "B", B, bc, dtype), *_step_rows(what, "C", C, bc, dtype),
                  *params, old,
                  old if out_state is None else _flat(what, "out_state", out_state, shape, f32),
                  0, *_NONE, *_NONE, *_NONE, *_NONE, *_NONE, *_NONE, 0, 0, 0, 0, 0)
    _call(what, u.device, _lib().canon_selective_scan_step, c)
    return out
