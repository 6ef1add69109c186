"""Checks of the sequence operators that need no GPU: exports, struct layout,
workspace sizes, and every refusal (no call here reaches a launch: each fails
validation, or has nothing to do)."""
import ctypes
import os
import re

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "canon_seq.h")
FAKE = 0x10000  # never dereferenced


@pytest.fixture(scope="module")
def seq():
    import scan_canonical_reduce_amd as c
    if not os.path.exists(c.LIB_PATH):
        from scan_canonical_reduce_amd import build
        build.build()
    from scan_canonical_reduce_amd import seq as s
    s._lib()
    return s


def header():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_header_exports(seq):
    names = sorted(set(re.findall(r"\b(canon_[a-z0-9_]+)\s*\(", header())))
    assert names == sorted(seq.SEQ_EXPORTS)
    out = os.popen(f"nm -D --defined-only {seq._lib()._name}").read()
    for name in names:
        assert re.search(rf"\bT {name}\b", out), name


class Rows(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("seq", ctypes.c_int64), ("row", ctypes.c_int64)]


def struct_of(name):
    """The header's struct as a ctypes one."""
    body = re.search(r"typedef struct \{([^}]*)\} " + name + ";", header()).group(1)
    fields = []
    for decl in filter(None, (d.strip() for d in body.split(";"))):
        kind, names = re.match(r"(?:const )?(\w+)(.*)", decl, re.S).groups()
        for n in names.split(","):
            c = ctypes.c_void_p if "*" in n else Rows if kind == "canon_rows_t" else ctypes.c_int64
            assert "*" in n or kind in ("canon_rows_t", "int64_t")
            fields.append((n.strip(" *\n"), c))
    return type(name, (ctypes.Structure,), {"_fields_": fields})


Conv, Scan = struct_of("canon_conv_t"), struct_of("canon_selective_scan_t")


def test_struct_sizes(seq):
    assert [f[0] for f in struct_of("canon_rows_t")._fields_] == ["p", "seq", "row"]
    assert ctypes.sizeof(Conv) == seq.CONV.size and ctypes.sizeof(Scan) == seq.SCAN.size


def test_limits_match_the_header(seq):
    text = header()
    for name, value in (("CANON_CONV_CHUNK", seq.CONV_CHUNK), ("CANON_SCAN_CHUNK", seq.SCAN_CHUNK),
                        ("CANON_MAX_STATES", seq.MAX_STATES), ("CANON_MAX_TAPS", seq.MAX_TAPS),
                        ("CANON_SEQ_VERSION", seq.SEQ_VERSION)):
        assert int(re.search(rf"#define {name} (\d+)", text).group(1)) == value
    assert seq._lib().canon_seq_version() == seq.SEQ_VERSION


def test_workspace_sizes(seq):
    w = seq.embedding_grad_workspace_bytes
    assert w(100, 0, 8) == 0 and w(100, 10, 0) == 0 and w(1 << 30, 10, 8) == 0
    assert w(100, 10, 8) % 256 == 0 and w(100, 10, 8) > 100 * 4 + 100 * 8
    assert w(0, 10, 8) > 0
    c = seq.causal_conv_grad_workspace_bytes
    assert c(1, 32, False, 64, 4) == (4 + 1) * 64 * 4
    assert c(1, 33, False, 64, 4) == 2 * (4 + 1) * 64 * 4
    assert c(3, 64, True, 64, 4) == 5 * (4 + 1) * 64 * 4
    assert c(1, 32, False, 64, 0) == 0 and c(1, 32, False, 64, 9) == 0
    s = seq.selective_scan_workspace_bytes
    assert s(2, 65, False, 64, 16) == 4 * 64 * (16 + 1) * 4
    assert s(2, 65, False, 64, 17) == 0 and s(2, 65, False, 64, 0) == 0
    g = seq.selective_scan_grad_workspace_bytes
    assert g(1, 64, False, 64, 1, 16) > s(1, 64, False, 64, 16)
    assert g(1, 64, False, 64, 3, 16) == 0 and g(1, 64, False, 64, 0, 16) == 0
    # large sizes do not wrap
    assert s(1, (1 << 30) - 1, False, (1 << 24) - 1, 16) > 1 << 50


def test_embedding_refusals(seq):
    L = seq._lib()

    def emb(dtype=1, w=FAKE, ld=8, rows=10, width=8, ids=FAKE, nb=8, tokens=4, out=FAKE, ldo=8):
        return L.canon_embedding(dtype, w, ld, rows, width, ids, nb, tokens, 1.0, out, ldo, None)

    for bad in (dict(dtype=3), dict(dtype=-1), dict(nb=2), dict(ld=7), dict(ldo=7),
                dict(w=None), dict(ids=None), dict(out=None)):
        assert emb(**bad) == 1, bad
    assert emb(tokens=0, ids=None, out=None) == 0
    assert emb(tokens=1 << 30) == 2 and emb(rows=1 << 31) == 2

    n = seq.embedding_grad_workspace_bytes(100, 10, 8)

    def grad(dtype=1, d=FAKE, ld=8, ids=FAKE, nb=8, tokens=100, rows=10, width=8, pad=-1, acc=0,
             gd=0, dw=FAKE, lw=8, ws=FAKE, wb=n):
        return L.canon_embedding_grad(dtype, d, ld, ids, nb, tokens, rows, width, 1.0, pad, acc,
                                      gd, dw, lw, ws, wb, None)

    for bad in (dict(dtype=3), dict(gd=2), dict(nb=1), dict(acc=2), dict(ld=7), dict(lw=7),
                dict(pad=-2), dict(dw=None), dict(ids=None), dict(d=None)):
        assert grad(**bad) == 1, bad
    for bad in (dict(ws=None), dict(wb=n - 1), dict(ws=FAKE + 8)):
        assert grad(**bad) == 3, bad
    assert grad(rows=0) == 0 and grad(width=0) == 0
    assert grad(tokens=1 << 30) == 2


def conv(seq, **kw):
    c = Conv()
    c.dtype, c.taps, c.silu, c.param_dtype = 1, 4, 1, 0
    c.seqs, c.rows, c.channels = 2, 9, 8
    r = Rows(FAKE, 72, 8)
    c.x = c.out = c.dout = c.dx = r
    c.weight = c.bias = c.dweight = c.dbias = FAKE
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


def test_conv_refusals(seq):
    L = seq._lib()
    n = seq.causal_conv_grad_workspace_bytes(2, 9, False, 8, 4)
    R = Rows
    for bad in (dict(dtype=7), dict(taps=0), dict(silu=2), dict(param_dtype=2), dict(seqs=-1),
                dict(rows=-1), dict(channels=-1), dict(weight=None), dict(x=R(None, 0, 0)),
                dict(x=R(FAKE, 72, -8))):
        assert L.canon_causal_conv(conv(seq, **bad), None) == 1, bad
        assert L.canon_causal_conv_grad(conv(seq, **bad), FAKE, n, None) == 1, bad
    for bad in (R(None, 0, 0), R(FAKE, 0, 8), R(FAKE, 72, 7), R(FAKE, 71, 8), R(FAKE, 8, 15)):
        assert L.canon_causal_conv(conv(seq, out=bad), None) == 1, (bad.seq, bad.row)
        assert L.canon_causal_conv_grad(conv(seq, dx=bad), FAKE, n, None) == 1
    assert L.canon_causal_conv(None, None) == 1
    for bad in (dict(taps=9), dict(rows=1 << 30), dict(channels=1 << 24)):
        assert L.canon_causal_conv(conv(seq, **bad), None) == 2, bad
    assert L.canon_causal_conv(conv(seq, rows=(1 << 30) - 1, seqs=1, channels=(1 << 24) - 1),
                               None) == 2
    assert L.canon_causal_conv_grad(conv(seq), FAKE, n - 1, None) == 3
    assert L.canon_causal_conv_grad(conv(seq), FAKE + 4, n, None) == 3
    assert L.canon_causal_conv_grad(conv(seq, dweight=None), FAKE, n, None) == 1
    assert L.canon_causal_conv_grad(conv(seq, bias=None), FAKE, n, None) == 1  # dbias, no bias
    assert L.canon_causal_conv_step(conv(seq, starts=FAKE), None) == 1
    assert L.canon_causal_conv(conv(seq, seqs=0, x=R(None, 0, 0)), None) == 0
    assert L.canon_causal_conv_step(conv(seq, channels=0), None) == 0


def scan(seq, **kw):
    c = Scan()
    c.dtype, c.softplus = 1, 1
    c.seqs, c.rows, c.channels, c.groups, c.states = 2, 9, 8, 2, 16
    r = Rows(FAKE, 72, 8)
    b = Rows(FAKE, 9 * 32, 32)
    c.u = c.delta = c.z = c.out = c.dout = c.du = c.ddelta = c.dz = r
    c.B = c.C = c.dB = c.dC = b
    c.A = c.D = c.delta_bias = c.dA = c.dD = c.ddelta_bias = c.chunk_states = FAKE
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


def test_scan_refusals(seq):
    L = seq._lib()
    R = Rows
    n = seq.selective_scan_grad_workspace_bytes(2, 9, False, 8, 2, 16)
    common = [dict(dtype=5), dict(softplus=2), dict(seqs=-1), dict(rows=-1), dict(groups=0),
              dict(groups=3), dict(states=0), dict(A=None), dict(u=R(None, 0, 0)),
              dict(delta=R(None, 0, 0)), dict(B=R(None, 0, 0)), dict(C=R(FAKE, -1, 1)),
              dict(z=R(FAKE, 72, -8)), dict(chunk_states=FAKE + 4)]
    for bad in common:
        assert L.canon_selective_scan(scan(seq, **bad), FAKE, n, None) == 1, bad
        assert L.canon_selective_scan_grad(scan(seq, **bad), FAKE, n, None) == 1, bad
    for bad in (R(None, 0, 0), R(FAKE, 0, 8), R(FAKE, 72, 7)):
        assert L.canon_selective_scan(scan(seq, out=bad), FAKE, n, None) == 1
        for name in ("du", "ddelta", "dz"):
            assert L.canon_selective_scan_grad(scan(seq, **{name: bad}), FAKE, n, None) == 1, name
    for name in ("dB", "dC"):
        assert L.canon_selective_scan_grad(scan(seq, **{name: R(FAKE, 9 * 32, 31)}), FAKE, n,
                                           None) == 1
    for bad in (dict(dA=None), dict(D=None), dict(delta_bias=None), dict(chunk_states=None),
                dict(channels=0, groups=1),
                dict(dout=R(None, 0, 0))):
        assert L.canon_selective_scan_grad(scan(seq, **bad), FAKE, n, None) == 1, bad
    for bad in (dict(states=17), dict(rows=1 << 30), dict(channels=1 << 24)):
        assert L.canon_selective_scan(scan(seq, **bad), FAKE, n, None) == 2, bad
    assert L.canon_selective_scan(scan(seq), FAKE, 255, None) == 3
    assert L.canon_selective_scan(scan(seq), None, 0, None) == 3
    assert L.canon_selective_scan_grad(scan(seq), FAKE, n - 1, None) == 3
    assert L.canon_selective_scan_step(scan(seq, starts=FAKE), None) == 1
    assert L.canon_selective_scan(None, FAKE, n, None) == 1
    assert L.canon_selective_scan(scan(seq, seqs=0, u=R(None, 0, 0)), None, 0, None) == 0
    assert L.canon_selective_scan_step(scan(seq, channels=0, groups=1), None) == 0


def test_the_binding_has_no_cpu_path(seq):
    import scan_canonical_reduce_amd as canon
    x, w = torch.zeros(1, 3, 8), torch.zeros(8, 4)
    A, B = torch.zeros(8, 16), torch.zeros(1, 3, 16)
    ids = torch.zeros(3, dtype=torch.int64)
    for call in (lambda: canon.embedding(w, ids), lambda: canon.embedding_grad(w[:3], ids, 9),
                 lambda: canon.causal_conv(x, w), lambda: canon.causal_conv_grad(x, x, w),
                 lambda: canon.causal_conv_step(x[0], x, w),
                 lambda: canon.selective_scan(x, x, A, B, B),
                 lambda: canon.selective_scan_grad(x, x, x, A, B, B, A),
                 lambda: canon.selective_scan_step(A[None], x[0], x[0], A, B[0], B[0])):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_no_sequences_need_no_workspace(seq):
    """Rows that belong to no sequence have no chunks."""
    for rows in (0, 64, 1000):
        for packed in (False, True):
            assert seq.causal_conv_grad_workspace_bytes(0, rows, packed, 64, 4) == 0
            assert seq.selective_scan_workspace_bytes(0, rows, packed, 64, 16) == 0
            assert seq._lib().canon_selective_scan_states(0, rows, int(packed), 64, 16) == 0


def test_backward_launch_limits(seq):
    """Two channels a thread in the convolution's backward pass, and the column
    sums of the parameters' gradients: launches below 2^32 threads."""
    L = seq._lib()
    r = Rows(FAKE, 4096, 4096)
    big = dict(seqs=5 << 19, rows=1, channels=4096, x=r, out=r, dout=r, dx=r)
    assert L.canon_causal_conv_grad(conv(seq, **big), None, 0, None) == 2
    n = 1 << 23
    r = Rows(FAKE, n, n)
    wide = dict(seqs=1, rows=1, channels=n, groups=1, u=r, delta=r, z=r, out=r, dout=r, du=r,
                ddelta=r, dz=r)
    assert L.canon_selective_scan_grad(scan(seq, **wide), None, 0, None) == 2
    assert L.canon_selective_scan(scan(seq, **wide), None, 0, None) == 3  # no workspace


def test_in_place_refusals(seq):
    """Outputs in an input's place, where that would read what it has written."""
    L = seq._lib()
    n = seq.causal_conv_grad_workspace_bytes(2, 9, False, 8, 4)
    x, y, z = (Rows(FAKE + i * 4096, 72, 8) for i in range(3))
    assert L.canon_causal_conv(conv(seq, x=x, out=x), None) == 1
    for a, b in ((x, z), (z, x)):
        assert L.canon_causal_conv_grad(conv(seq, x=a, dout=b, dx=x), FAKE, n, None) == 1
    assert L.canon_causal_conv_grad(conv(seq, x=x, dout=y, dx=z), FAKE, n - 1, None) == 3
    assert L.canon_embedding(1, FAKE, 8, 10, 8, FAKE, 8, 4, 1.0, FAKE, 8, None) == 1
    m = seq.embedding_grad_workspace_bytes(100, 10, 8)
    assert L.canon_embedding_grad(1, FAKE, 8, FAKE, 8, 100, 10, 8, 1.0, -1, 0, 0, FAKE, 8, FAKE,
                                  m, None) == 1


def test_limits_of_a_launch(seq):
    """The header's limits at their edges: one step beyond is refused, at the edge a
    call comes as far as the workspace that it is not given."""
    L = seq._lib()

    def emb(dtype, tokens, width):
        return L.canon_embedding(dtype, FAKE, width, 10, width, FAKE, 8, tokens, 1.0, FAKE + 16,
                                 width, None)

    # 2^34 accesses of 16 bytes, and of single elements
    assert emb(1, 1 << 25, 4096) == 2 and emb(0, 1 << 25, 2048) == 2
    assert emb(1, (1 << 34) // 513 + 1, 4097) == 2
    assert emb(1, 1 << 29, 1 << 10) == 2

    def rows(n):
        return Rows(FAKE, n, n)

    def conv_grad(channels, seqs):
        r = rows(channels)
        return L.canon_causal_conv_grad(conv(seq, seqs=seqs, rows=1, channels=channels, x=r, out=r,
                                             dout=r, dx=Rows(FAKE + 8, channels, channels)),
                                        None, 0, None)

    most = (1 << 32) - (1 << 24)
    assert conv_grad(8192, most // 4096) == 3 and conv_grad(8192, most // 4096 + 1) == 2
    assert conv_grad(8191, most // 8191) == 3 and conv_grad(8191, most // 8191 + 1) == 2

    def scan_grad(channels, groups, states, seqs, n=1):
        r, b = Rows(FAKE, n * channels, channels), Rows(FAKE, n * groups * states, groups * states)
        return L.canon_selective_scan_grad(
            scan(seq, channels=channels, groups=groups, states=states, seqs=seqs, rows=n, u=r,
                 delta=r, z=r, out=r, dout=r, du=r, ddelta=r, dz=r, B=b, C=b, dB=b, dC=b),
            None, 0, None)

    # rows of all sequences x groups x padded states
    for groups, states, padded in ((1, 16, 16), (2, 13, 16), (4, 7, 8), (1, 3, 4)):
        n = (1 << 30) // (groups * padded)
        assert scan_grad(64, groups, states, n // 64, 64) == 3
        assert scan_grad(64, groups, states, n // 64 + 1, 64) == 2
    # chunks x slabs
    assert scan_grad(130, 1, 1, ((1 << 24) - 1) // 3) == 3
    assert scan_grad(130, 1, 1, ((1 << 24) - 1) // 3 + 1) == 2
    # columns of the parameters' sums
    edge = (1 << 26) // 18
    assert scan_grad(edge, 1, 16, 1) == 3 and scan_grad(edge + 1, 1, 16, 1) == 2


def test_rows_of_the_largest_gradient(seq):
    """Above 2^31 - 512 rows the grouping kernel would need 2^22 workgroups of 1024
    threads: refused, whatever the number of tokens."""
    L = seq._lib()
    for rows, status in (((1 << 31) - 512, 3), ((1 << 31) - 511, 2), ((1 << 31) - 1, 2)):
        for tokens in (0, 1, 1000, 5000):
            assert L.canon_embedding_grad(1, FAKE, 8, FAKE, 8, tokens, rows, 8, 1.0, -1, 0, 0, FAKE,
                                          8, None, 0, None) == status, (rows, tokens)
        assert (seq.embedding_grad_workspace_bytes(5000, rows, 8) > 0) == (status == 3)
