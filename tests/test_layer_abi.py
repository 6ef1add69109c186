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


Norm = struct_of("canon_norm_t")


def layout(struct):
    """The struct's fields as the binding packs them."""
    code = {Rows: "qqq", ctypes.c_double: "d"}
    return "".join(code.get(t, "q") for _, t in struct._fields_)


def test_struct_layouts(layer):
    def spelt(s):
        return re.sub(r"(\d+)(\w)", lambda m: m.group(2) * int(m.group(1)), s.format.lstrip("="))

    assert spelt(layer.NORM) == layout(Norm) and layer.NORM.size == ctypes.sizeof(Norm)


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
    """Backward: chunks of rows times column tiles below 2^24."""
    L, n = layer._lib(), (1 << 24) - 1
    wide = Rows(FAKE, n, n)
    out = Rows(FAKE + 512, n, n)
    rows = 64 * 1023
    assert L.canon_layer_norm_grad(norm(seqs=1, rows=rows, width=n, x=wide, dout=wide, dsum=wide,
                                        dx=out), None, 0, None) == 3
    assert L.canon_layer_norm_grad(norm(seqs=1, rows=rows + 64, width=n, x=wide, dout=wide,
                                        dsum=wide, dx=out), None, 0, None) == 2


def test_the_binding_has_no_cpu_path(layer):
    import scan_canonical_reduce_amd as canon
    x, w = torch.zeros(3, 8), torch.ones(8)
    for call in (lambda: canon.layer_norm(x, w), lambda: canon.add_layer_norm(x, x, w),
                 lambda: canon.layer_norm_grad(x, x, w, canon.layer_norm_stats(x))):
        with pytest.raises(ValueError, match="GPU"):
            call()
