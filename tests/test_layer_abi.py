"""Checks of the layer operators that need no GPU: exports, struct layout, workspace
sizes, and every refusal (no call here reaches a launch: each fails validation, or
has nothing to do)."""
import ctypes
import os
import re

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "canon_layer.h")
FAKE = 0x10000  # never dereferenced


@pytest.fixture(scope="module")
def layer():
    import scan_canonical_reduce_amd as c
    if not os.path.exists(c.LIB_PATH):
        from scan_canonical_reduce_amd import build
        build.build()
    from scan_canonical_reduce_amd import layer as m
    m._lib()
    return m


def header():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_header_exports(layer):
    names = sorted(set(re.findall(r"\b(canon_[a-z0-9_]+)\s*\(", header())))
    assert names == sorted(layer.LAYER_EXPORTS)
    out = os.popen(f"nm -D --defined-only {layer._lib()._name}").read()
    for name in names:
        assert re.search(rf"\bT {name}\b", out), name
    assert layer._lib().canon_layer_version() == layer.LAYER_VERSION
    assert int(re.search(r"#define CANON_LAYER_VERSION (\d+)", header()).group(1)) == \
        layer.LAYER_VERSION


class Rows(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("seq", ctypes.c_int64), ("row", ctypes.c_int64)]


def struct_of(name):
    """The header's struct as a ctypes one."""
    body = re.search(r"typedef struct \{([^}]*)\} " + name + ";", header()).group(1)
    kinds = {"canon_rows_t": Rows, "int64_t": ctypes.c_int64, "double": ctypes.c_double}
    fields = []
    for decl in filter(None, (d.strip() for d in body.split(";"))):
        kind, names = re.match(r"(?:const )?(\w+)(.*)", decl, re.S).groups()
        for n in names.split(","):
            fields.append((n.strip(" *\n"), ctypes.c_void_p if "*" in n else kinds[kind]))
    return type(name, (ctypes.Structure,), {"_fields_": fields})


Norm, Recur = struct_of("canon_norm_t"), struct_of("canon_recur_t")
Sample = struct_of("canon_sample_t")


def layout(struct):
    """The struct's fields as the binding packs them."""
    code = {Rows: "qqq", ctypes.c_double: "d"}
    return "".join(code.get(t, "q") for _, t in struct._fields_)


def test_struct_layouts(layer):
    def spelt(s):
        return re.sub(r"(\d+)(\w)", lambda m: m.group(2) * int(m.group(1)), s.format.lstrip("="))

    for packed, struct in ((layer.NORM, Norm), (layer.RECUR, Recur),
                           (layer.SAMPLE, Sample)):
        assert spelt(packed) == layout(struct) and packed.size == ctypes.sizeof(struct)


def norm(**kw):
    c = Norm()
    c.dtype, c.param_dtype, c.seqs, c.rows, c.width, c.eps = 1, 0, 2, 9, 8, 1e-5
    at = iter(range(2 * FAKE, 3 * FAKE, 4096))
    for k in ("x", "residual", "sum", "out", "dout", "dsum", "dx"):
        setattr(c, k, Rows(next(at), 72, 8))
    c.weight = c.bias = c.stats = c.dweight = c.dbias = FAKE
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


def test_norm_workspace(layer):
    w = layer.layer_norm_grad_workspace_bytes
    assert w(1, 0, 8) == 0 and w(1, 1, 64) == 2 * 256 and w(2, 9, 64) == 2 * 18 * 256
    assert w(1, 512, 64) == 2 * 512 * 256 and w(1, 513, 64) == 2 * 257 * 256
    assert w(1, 1 << 20, 64) == 2 * (1 << 14) * 256
    assert w(1 << 30, 1, 8) == 0 and w(1 << 16, 1 << 15, 8) == 0 and w(1, 1, 1 << 24) == 0


def test_norm_refusals(layer):
    L, R = layer._lib(), Rows
    n = layer.layer_norm_grad_workspace_bytes(2, 9, 8)
    for bad in (dict(dtype=3), dict(param_dtype=2), dict(seqs=-1), dict(rows=-1), dict(width=-1),
                dict(weight=None), dict(x=R(None, 0, 0)), dict(x=R(FAKE, 72, -8))):
        assert L.canon_layer_norm(norm(**bad), None) == 1, bad
        assert L.canon_layer_norm_grad(norm(**bad), FAKE, n, None) == 1, bad
    for bad in (R(None, 0, 0), R(FAKE + 512, 0, 8), R(FAKE + 512, 72, 7), R(FAKE + 512, 71, 8)):
        assert L.canon_layer_norm(norm(out=bad), None) == 1
        assert L.canon_layer_norm_grad(norm(dx=bad), FAKE, n, None) == 1
    assert L.canon_layer_norm(norm(sum=R(FAKE + 512, 72, 7)), None) == 1
    assert L.canon_layer_norm(norm(residual=R(None, 0, 0)), None) == 1  # a sum of one
    for bad in (dict(dout=R(None, 0, 0)), dict(dsum=R(FAKE, -1, 8)), dict(stats=None),
                dict(dweight=None)):
        assert L.canon_layer_norm_grad(norm(**bad), FAKE, n, None) == 1, bad
    for bad in (dict(seqs=1 << 30), dict(rows=1 << 30), dict(width=1 << 24),
                dict(seqs=1 << 16, rows=1 << 15)):
        assert L.canon_layer_norm(norm(**bad), None) == 2, bad
        assert L.canon_layer_norm_grad(norm(**bad), FAKE, n, None) == 2, bad
    assert L.canon_layer_norm_grad(norm(), FAKE, n - 1, None) == 3
    assert L.canon_layer_norm_grad(norm(), FAKE + 8, n, None) == 3
    assert L.canon_layer_norm(None, None) == 1 and L.canon_layer_norm_grad(None, FAKE, n, None) == 1
    for none in (dict(seqs=0), dict(rows=0), dict(width=0)):
        assert L.canon_layer_norm(norm(x=R(None, 0, 0), out=R(None, 0, 0), **none), None) == 0
    assert L.canon_layer_norm_grad(norm(width=0, dweight=None), None, 0, None) == 0


def test_norm_in_place(layer):
    """Outputs in an input's place: the same elements only, and not where a later step
    reads the input."""
    L, R = layer._lib(), Rows
    n = layer.layer_norm_grad_workspace_bytes(2, 9, 8)
    x = R(FAKE, 72, 8)
    shifted = R(FAKE, 200, 16)
    assert L.canon_layer_norm(norm(x=x, out=shifted), None) == 1
    assert L.canon_layer_norm(norm(residual=x, out=shifted), None) == 1
    assert L.canon_layer_norm(norm(residual=x, sum=shifted), None) == 1
    assert L.canon_layer_norm(norm(sum=x, out=x), None) == 1
    assert L.canon_layer_norm_grad(norm(x=x, dx=x), FAKE, n, None) == 1
    assert L.canon_layer_norm_grad(norm(dout=x, dx=shifted), FAKE, n, None) == 1
    assert L.canon_layer_norm_grad(norm(dsum=x, dx=shifted), FAKE, n, None) == 1
    assert L.canon_layer_norm_grad(norm(dout=x, dx=x), FAKE, n - 1, None) == 3


def test_norm_launch_limits(layer):
    """Rows of all sequences below 2^30; backward: chunks of rows times column tiles
    below 2^24."""
    L, n = layer._lib(), (1 << 24) - 1
    for seqs, rows, want in ((1 << 15, (1 << 15) - 1, 3), (1 << 15, 1 << 15, 2),
                             ((1 << 30) - 128, 1, 3), (2, 1 << 29, 2)):
        x, out = Rows(FAKE, rows, 1), Rows(FAKE + 512, rows, 1)
        kw = dict(seqs=seqs, rows=rows, width=1, x=x, dout=x, dsum=x, dx=out)
        assert L.canon_layer_norm_grad(norm(**kw), None, 0, None) == want
        assert (L.canon_layer_norm_grad_workspace_bytes(seqs, rows, 1) == 0) == (want == 2)
        if want == 2:
            assert L.canon_layer_norm(norm(**dict(kw, residual=x, sum=out, out=out)), None) == 2
    wide = Rows(FAKE, n, n)
    out = Rows(FAKE + 512, n, n)
    rows = 64 * 1023
    assert L.canon_layer_norm_grad(norm(seqs=1, rows=rows, width=n, x=wide, dout=wide, dsum=wide,
                                        dx=out), None, 0, None) == 3
    assert L.canon_layer_norm_grad(norm(seqs=1, rows=rows + 64, width=n, x=wide, dout=wide,
                                        dsum=wide, dx=out), None, 0, None) == 2


def recur(**kw):
    c = Recur()
    c.dtype, c.seqs, c.rows, c.channels = 1, 2, 9, 8
    at = iter(range(2 * FAKE, 3 * FAKE, 4096))
    for k in ("x", "gate", "input_gate", "out", "dout", "dx", "dgate", "dinput_gate"):
        setattr(c, k, Rows(next(at), 72, 8))
    c.decay = c.ddecay = c.kept_states = FAKE
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


def test_recur_workspace(layer):
    w, g = layer.gated_recurrence_workspace_bytes, layer.gated_recurrence_grad_workspace_bytes
    s = layer._lib().canon_gated_recurrence_states
    # a workgroup for each round (of up to 64 slots of 64 channels, 128 where sequences
    # have 2 to 15 blocks): two folds of each of 64 chunks a slot, and the start states
    assert w(3, 256, False, 64) == 0 and g(3, 256, False, 64) == 3 * 256
    assert w(3, 257, False, 64) == 3 * 129 * 256 and g(3, 257, False, 64) == 3 * 132 * 256
    assert w(64, 512, False, 64) == 64 * 129 * 256 and w(65, 512, False, 64) == 0
    assert w(64, 513, False, 64) == 128 * 129 * 256 and w(65, 513, False, 64) == 3 * 130 * 256
    assert w(3, 1024, True, 64) == 5 * 129 * 256
    assert w(1, 15 * 512, False, 64) == 15 * 129 * 256
    assert w(1, 15 * 512 + 1, False, 64) == 3 * 16 * 256
    # two folds and the start state of each block
    assert w(200, 513, False, 64) == 3 * 400 * 256 and g(200, 513, False, 64) == 4 * 400 * 256
    assert w(200, 1024, True, 64) == 3 * 202 * 256 and w(200, 512, True, 64) == 0
    assert s(3, 513, 0, 64) == 6 * 4 * 64 and s(3, 1024, 1, 64) == 5 * 4 * 64
    assert w(0, 1024, True, 64) == 0 and g(0, 1024, True, 64) == 0 and s(0, 99, 1, 64) == 0
    for bad in ((1 << 30, 1, False, 8), (1, 1 << 30, False, 8), (1, 1, False, 1 << 24)):
        assert w(*bad) == 0 and g(*bad) == 0 and s(*bad) == 0
    assert w(1, (1 << 30) - 1, False, (1 << 24) - 1) > 1 << 46  # large sizes do not wrap


def test_recur_refusals(layer):
    L, R = layer._lib(), Rows
    n = layer.gated_recurrence_grad_workspace_bytes(2, 9, False, 8)
    calls = (lambda **b: L.canon_gated_recurrence(recur(**b), None, 0, None),
             lambda **b: L.canon_gated_recurrence_grad(recur(**b), FAKE, n, None))
    step = lambda **b: L.canon_gated_recurrence_step(recur(**b), None)  # noqa: E731
    for bad in (dict(dtype=3), dict(seqs=-1), dict(rows=-1), dict(channels=-1),
                dict(x=R(None, 0, 0)), dict(gate=R(None, 0, 0)), dict(gate=R(FAKE, -1, 8)),
                dict(input_gate=R(FAKE, 72, -8))):
        assert all(call(**bad) == 1 for call in calls), bad
    for bad in (R(None, 0, 0), R(FAKE, 0, 8), R(FAKE, 72, 7), R(FAKE, 71, 8)):
        assert calls[0](out=bad) == 1
        for name in ("dx", "dgate", "dinput_gate"):
            assert calls[1](**{name: bad}) == 1, name
    x = R(2 * FAKE, 72, 8)
    for name in ("x", "gate", "input_gate"):  # in place
        assert calls[0](**{name: x, "out": x}) == 1
    for name in ("x", "gate", "input_gate", "dout"):
        for out in ("dx", "dgate", "dinput_gate"):
            assert calls[1](**{name: x, out: x}) == 1, (name, out)
    assert calls[1](dx=x, dgate=x) == 1 and calls[1](dx=x, dinput_gate=x) == 1
    for bad in (dict(dout=R(None, 0, 0)), dict(kept_states=None), dict(ddecay=None),
                dict(decay=None), dict(d_init_state=FAKE, d_final_state=FAKE)):
        assert calls[1](**bad) == 1, bad
    for bad in (dict(rows=1 << 30), dict(seqs=1 << 30), dict(channels=1 << 24)):
        assert all(call(**bad) == 2 for call in calls), bad
    assert L.canon_gated_recurrence(recur(rows=513, x=R(FAKE, 513 * 8, 8),
                                          out=R(3 * FAKE, 513 * 8, 8)), None, 0, None) == 3
    assert L.canon_gated_recurrence_grad(recur(), FAKE, n - 1, None) == 3
    assert L.canon_gated_recurrence_grad(recur(), FAKE + 8, n, None) == 3
    assert step(starts=FAKE) == 1 and step(x=R(None, 0, 0)) == 1
    assert L.canon_gated_recurrence(None, None, 0, None) == 1
    assert L.canon_gated_recurrence_grad(None, None, 0, None) == 1
    assert L.canon_gated_recurrence_step(None, None) == 1
    for none in (dict(seqs=0), dict(channels=0)):
        assert calls[0](x=R(None, 0, 0), **none) == 0 and step(x=R(None, 0, 0), **none) == 0
    assert calls[1](channels=0, x=R(None, 0, 0)) == 0


def test_recur_launch_limits(layer):
    """Blocks times slabs below 2^22."""
    L = layer._lib()

    def call(seqs, rows, channels, **kw):
        r = Rows(FAKE, rows * channels, channels)
        return L.canon_gated_recurrence(recur(seqs=seqs, rows=rows, channels=channels, x=r, gate=r,
                                              input_gate=r,
                                              out=Rows(3 * FAKE, rows * channels, channels), **kw),
                                        None, 0, None)

    assert call((1 << 21) - 1, 513, 64) == 3 and call(1 << 21, 513, 64) == 2
    most = ((1 << 22) - 1) // 16383  # channels of 16383 slabs
    assert call(1, 512 * most, 64 * 16383) == 3 and call(1, 512 * most + 1, 64 * 16383) == 2
    p = dict(starts=FAKE)
    assert call(1, 512 * most - 1, 64 * 16383, **p) == 3
    assert call(1, 512 * most, 64 * 16383, **p) == 2
    # row pitches, but for single rows
    wide = 1 << 24
    for name in ("x", "gate", "input_gate", "out"):
        ok, far = ({name: Rows(FAKE * (3 if name == "out" else 1), 600 * p, p)}
                   for p in (wide - 1, wide))
        c = dict(seqs=1, rows=600, channels=64, x=Rows(FAKE, 64 * 600, 64),
                 gate=Rows(FAKE, 64 * 600, 64), input_gate=Rows(FAKE, 64 * 600, 64),
                 out=Rows(3 * FAKE, 64 * 600, 64))
        assert L.canon_gated_recurrence(recur(**{**c, **ok}), None, 0, None) == 3, name
        assert L.canon_gated_recurrence(recur(**{**c, **far}), None, 0, None) == 2, name
    r = Rows(FAKE, 64, 64)
    assert L.canon_gated_recurrence_step(recur(seqs=1 << 22, channels=64, x=r, gate=r, input_gate=r,
                                               out=Rows(3 * FAKE, 64, 64)), None) == 2


def sample(**kw):
    c = Sample()
    c.dtype, c.rows, c.vocab, c.ld, c.id_bytes = 0, 3, 50, 50, 8
    c.logits = c.u = c.ids = FAKE
    c.temperature_all, c.top_p_all = 1.0, 1.0
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


def test_sample_refusals(layer):
    L = layer._lib()
    ws = layer.sample_workspace_bytes
    for bad in (dict(dtype=3), dict(rows=-1), dict(vocab=-1), dict(ld=-1), dict(id_bytes=2),
                dict(logits=None), dict(u=None), dict(ids=None)):
        assert L.canon_sample(sample(**bad), FAKE, ws(3, 50), None) == 1, bad
    assert L.canon_sample(None, FAKE, 0, None) == 1
    assert L.canon_sample(sample(rows=1 << 22), FAKE, 0, None) == 2
    assert L.canon_sample(sample(vocab=1 << 24), FAKE, 0, None) == 2
    assert L.canon_sample(sample(rows=0, ids=None, u=None, logits=None), None, 0, None) == 0


def test_the_binding_has_no_cpu_path(layer):
    import scan_canonical_reduce_amd as canon
    x, w = torch.zeros(3, 8), torch.ones(8)
    for call in (lambda: canon.layer_norm(x, w), lambda: canon.add_layer_norm(x, x, w),
                 lambda: canon.layer_norm_grad(x, x, w, canon.layer_norm_stats(x)),
                 lambda: canon.gated_recurrence(x[None], x[None]),
                 lambda: canon.sample(x, w),
                 lambda: canon.gated_recurrence_grad(x[None], x[None], x[None], w),
                 lambda: canon.gated_recurrence_step(x, x, x)):
        with pytest.raises(ValueError, match="GPU"):
            call()
