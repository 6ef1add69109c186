"""Embedding lookup and its gradient: bit for bit against the float32
expressions (the gradient's sums by the oracle's pairwise tree)."""
import numpy as np
import pytest

import oracle
from gpu_util import launches

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def canon():
    import scan_canonical_reduce_amd as c
    return c


def same_bits(a, b):
    ai = a.contiguous().view(torch.int32 if a.dtype == F32 else torch.int16)
    bi = b.contiguous().view(torch.int32 if b.dtype == F32 else torch.int16)
    return bool((ai.cpu() == bi.cpu()).all())


def make_ids(n, rows, kind, seed, dtype=torch.int64):
    g = torch.Generator().manual_seed(seed)
    if kind == "one":
        ids = torch.full((n,), rows // 2)
    elif kind == "few":
        ids = torch.randint(0, min(rows, 3), (n,), generator=g)
    else:
        ids = torch.exp(torch.rand(n, generator=g, dtype=torch.float64)
                        * np.log(rows)).long().clamp(1, rows) - 1
    if kind == "stray":  # outside the table on both sides
        stray = torch.rand(n, generator=g)
        ids[stray < 0.2] = -1
        ids[stray > 0.9] = rows
    return ids.to(dtype)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("width", [1, 7, 8, 250, 1000, 4096])
@pytest.mark.parametrize("ids_dtype", [torch.int64, torch.int32])
def test_lookup(canon, dtype, width, ids_dtype):
    rows, n = 131, 77
    w = torch.randn(rows, width, generator=torch.Generator().manual_seed(width)).to(dtype)
    ids = make_ids(n, rows, "stray", width, ids_dtype)
    ok = (ids >= 0) & (ids < rows)
    for scale in (1.0, 8.0, 1.7):
        want = (w[torch.where(ok, ids, 0).long()].float() * scale) * ok[:, None]
        got = canon.embedding(w.cuda(), ids.cuda(), scale=scale)
        assert torch.equal(got.cpu(), want.to(dtype)), scale


def test_lookup_shapes_strides_and_extremes(canon):
    w = torch.randn(50, 96)
    big = w.cuda()
    ids = torch.tensor([[3, 49], [0, 0], [-2 ** 31, 2 ** 31 - 1]], dtype=torch.int32).cuda()
    got = canon.embedding(big[:, 16:80], ids)  # pitch 96, offset 16 elements
    assert got.shape == (3, 2, 64)
    assert torch.equal(got[0].cpu(), w[[3, 49], 16:80]) and not got[2].any()
    out = torch.full((4, 80), 7.0, device="cuda")
    canon.embedding(big[:, 1:65], ids.view(-1)[:4], out=out[:, 3:67])  # no alignment
    assert torch.equal(out[:, 3:67].cpu(), w[[3, 49, 0, 0], 1:65])
    assert (out[:, :3] == 7).all() and (out[:, 67:] == 7).all()
    far = torch.tensor([2 ** 62, -2 ** 63, 2 ** 32 + 3, 3], device="cuda")
    got = canon.embedding(big, far)
    assert not got[:3].any() and torch.equal(got[3].cpu(), w[3])
    special = torch.tensor([[float("inf"), float("-inf"), float("nan"), -0.0]]).cuda()
    got = canon.embedding(special, torch.zeros(2, dtype=torch.int64, device="cuda"))
    assert got[1, 0] == float("inf") and got[1, 1] == float("-inf") and torch.isnan(got[1, 2])
    for shape in ((0,), (0, 3)):
        assert canon.embedding(big, torch.zeros(shape, dtype=torch.int64,
                                                device="cuda")).shape == shape + (96,)
    assert not canon.embedding(torch.empty(0, 8, device="cuda"),
                               torch.zeros(3, dtype=torch.int64, device="cuda")).any()


def grad_ref(dout, ids, rows, scale, padding=None, old=None, dtype=F32):
    x = dout.float().numpy()
    dw = torch.zeros(rows, x.shape[1]) if old is None else old.float().clone()
    for v in sorted(set(ids.tolist())):
        if v < 0 or v >= rows or v == padding:
            continue
        seg = np.ascontiguousarray(x[np.nonzero(ids.numpy() == v)[0]].T)
        r = torch.from_numpy(np.asarray(oracle.reduce_rows(seg, 1, -0.0), np.float32)) * scale
        dw[v] = r if old is None else dw[v] + r
    return dw.to(dtype)


@pytest.mark.parametrize("tokens,rows,width,kind", [
    (1, 1, 1, "zipf"), (1, 70000, 8, "zipf"), (63, 17, 24, "one"), (64, 17, 24, "one"),
    (65, 17, 24, "one"), (127, 5, 9, "few"), (128, 5, 8, "one"), (129, 5, 8, "one"),
    (1000, 513, 130, "zipf"), (3001, 10007, 40, "stray"), (5000, 300, 520, "few"),
    (4096, 16, 16, "one"), (9000, 2, 3, "few"), (70000, 40, 4, "few"), (2500, 140001, 64, "zipf"),
    (300, 600000, 4, "stray"),
])
@pytest.mark.parametrize("dtype,grad", [(F32, F32), (BF16, F32), (BF16, BF16), (F16, F16)])
def test_grad(canon, tokens, rows, width, kind, dtype, grad):
    dout = torch.randn(tokens, width, generator=torch.Generator().manual_seed(tokens)).to(dtype)
    ids = make_ids(tokens, rows, kind, rows)
    got = canon.embedding_grad(dout.cuda(), ids.cuda(), rows, scale=1.7, dtype=grad)
    assert got.dtype == grad
    assert same_bits(got, grad_ref(dout, ids, rows, np.float32(1.7).item(), dtype=grad))


@pytest.mark.parametrize("grad", [F32, BF16])
def test_grad_accumulate_and_padding(canon, grad):
    dout = torch.randn(700, 96).to(BF16)
    ids = make_ids(700, 90, "zipf", 3, torch.int32)
    old = torch.randn(90, 96).to(grad)
    out = old.cuda()
    got = canon.embedding_grad(dout.cuda(), ids.cuda(), 90, scale=0.5, padding_id=0, out=out,
                               accumulate=True)
    assert got is out
    want = grad_ref(dout, ids, 90, 0.5, 0, old, grad)
    assert same_bits(got, want)
    assert same_bits(got[0], old[0])  # the padding id: frequent, and untouched
    fresh = canon.embedding_grad(dout.cuda(), ids.cuda(), 90, scale=0.5, padding_id=0, dtype=grad)
    assert not fresh[0].any()


def test_grad_strides_empty_and_workspace(canon):
    dout = torch.randn(200, 64)
    ids = make_ids(200, 33, "zipf", 5)
    want = grad_ref(dout[:, 5:45], ids, 33, 1.0)
    out = torch.full((33, 50), 7.0, device="cuda")
    n = canon.embedding_grad_workspace_bytes(200, 33, 40)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(2):  # a workspace's contents do not matter
        canon.embedding_grad(dout.cuda()[:, 5:45], ids.cuda(), 33, out=out[:, 7:47], ws=ws)
        assert same_bits(out[:, 7:47], want)
        assert (out[:, :7] == 7).all() and (out[:, 47:] == 7).all()
    none = canon.embedding_grad(torch.empty(0, 8, device="cuda"),
                                torch.empty(0, dtype=torch.int64, device="cuda"), 9)
    assert none.shape == (9, 8) and not none.any()
    keep = torch.ones(9, 8, device="cuda")
    canon.embedding_grad(torch.ones(3, 8, device="cuda"),
                         torch.full((3,), -1, device="cuda"), 9, out=keep, accumulate=True)
    assert (keep == 1).all()
    assert canon.embedding_grad(torch.empty(3, 0, device="cuda"),
                                torch.zeros(3, dtype=torch.int64, device="cuda"), 9).numel() == 0


def test_grad_special_values(canon):
    """A NaN or an infinity reaches its own row and column alone; -0 sums to -0."""
    dout = torch.zeros(300, 16) - 0.0
    dout[7, 3], dout[8, 4], dout[250, 5] = float("nan"), float("inf"), float("-inf")
    ids = torch.arange(300) % 3
    got = canon.embedding_grad(dout.cuda(), ids.cuda(), 4)
    want = grad_ref(dout, ids, 4, 1.0)
    assert torch.equal(torch.isnan(got).cpu(), torch.isnan(want))
    ok = ~torch.isnan(want)
    assert torch.equal(got.cpu()[ok].view(torch.int32), want[ok].view(torch.int32))


def test_grad_does_not_depend_on_the_schedule(canon):
    dout = torch.randn(4000, 520, device="cuda")
    ids = make_ids(4000, 50, "zipf", 9).cuda()
    want = canon.embedding_grad(dout, ids, 50)
    for grid in (1, 3, 64):
        with canon.schedule(grid=grid):
            assert same_bits(canon.embedding_grad(dout, ids, 50), want)


def test_refusals(canon):
    w = torch.randn(10, 8, device="cuda")
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    with pytest.raises(TypeError):
        canon.embedding(w.double(), ids)
    with pytest.raises(ValueError):
        canon.embedding(w, ids.float())
    with pytest.raises(ValueError):
        canon.embedding(w.t(), ids)
    with pytest.raises(ValueError):
        canon.embedding(w, ids, out=torch.empty(4, 9, device="cuda"))
    with pytest.raises(ValueError):
        canon.embedding(w, ids.cpu())
    with pytest.raises(ValueError):
        canon.embedding_grad(w[:3], ids, 10)
    with pytest.raises(ValueError):
        canon.embedding_grad(w[:4], ids, 10, accumulate=True)
    with pytest.raises(ValueError):
        canon.embedding_grad(w[:4], ids, 10, padding_id=-3)
    with pytest.raises(TypeError):
        canon.embedding_grad(w[:4], ids, 10, dtype=torch.float16)
    with pytest.raises(ValueError):
        canon.embedding_grad(w[:4], ids, 10, out=torch.empty(9, 8, device="cuda"))


@pytest.mark.parametrize("dtype,grad", [(F32, F32), (BF16, F32), (BF16, BF16), (F16, F16)])
@pytest.mark.parametrize("width", [3, 4, 5, 7, 8, 9, 15, 63, 515, 1001])
def test_rows_of_any_width_and_place(canon, dtype, grad, width):
    """Rows that are not whole 16-byte vectors, or not aligned to them: same bits,
    each column added once, nothing written beside the rows."""
    g = torch.Generator().manual_seed(width)
    table = torch.randn(40, width + 9, generator=g).to(dtype).cuda()
    for tokens, off, kind in ((3, 0, "zipf"), (200, 1, "few"), (900, 0, "zipf"), (900, 3, "one")):
        ids = make_ids(tokens, 40, kind, tokens)
        w = table[:, off:off + width]
        out = torch.full((tokens, width + 4), 7.0, dtype=dtype, device="cuda")
        canon.embedding(w, ids.cuda(), 0.5, out=out[:, off:off + width])
        assert same_bits(out[:, off:off + width], (w.float() * 0.5)[ids.cuda()].to(dtype))
        assert (out[:, :off] == 7).all() and (out[:, off + width:] == 7).all()
        dout = torch.randn(tokens, width + 5, generator=g).to(dtype)[:, off:off + width]
        dw = torch.full((40, width + 4), 7.0, dtype=grad, device="cuda")
        canon.embedding_grad(dout.cuda(), ids.cuda(), 40, 1.5, out=dw[:, off:off + width])
        assert same_bits(dw[:, off:off + width], grad_ref(dout, ids, 40, 1.5, dtype=grad))
        old = dw[:, off:off + width].cpu()
        canon.embedding_grad(dout.cuda(), ids.cuda(), 40, 1.5, out=dw[:, off:off + width],
                             accumulate=True)
        assert same_bits(dw[:, off:off + width], grad_ref(dout, ids, 40, 1.5, None, old, grad))
        assert (dw[:, :off] == 7).all() and (dw[:, off + width:] == 7).all()


@pytest.mark.parametrize("tokens", [257, 1000, 4096])
@pytest.mark.parametrize("rows,width,off", [(256, 2056, 0), (300, 1001, 1), (3000, 130, 0),
                                            (3000, 3, 0), (140001, 8, 0), (5000, 520, 0)])
def test_grad_of_some_thousand_tokens(canon, tokens, rows, width, off):
    g = torch.Generator().manual_seed(tokens + width)
    dout = torch.randn(tokens, width + 8, generator=g).to(BF16)[:, off:off + width]
    ws = torch.full((canon.embedding_grad_workspace_bytes(tokens, rows, width),), 255,
                    dtype=torch.uint8, device="cuda")  # NaN wherever it is not written
    for kind, grad in (("zipf", F32), ("one", BF16), ("stray", BF16), ("few", F32)):
        ids = make_ids(tokens, rows, kind, tokens)
        dw = torch.full((rows, width + 8), 7.0, dtype=grad, device="cuda")
        got = dw[:, off:off + width]
        canon.embedding_grad(dout.cuda(), ids.cuda(), rows, 0.75, padding_id=2, out=got, ws=ws)
        want = grad_ref(dout, ids, rows, 0.75, 2, dtype=grad)
        assert same_bits(got, want), kind
        canon.embedding_grad(dout.cuda(), ids.int().cuda(), rows, 0.75, padding_id=2, out=got,
                             accumulate=True, ws=ws)
        assert same_bits(got, grad_ref(dout, ids, rows, 0.75, 2, want, grad)), kind
        assert (dw[:, :off] == 7).all() and (dw[:, off + width:] == 7).all()


def test_lookup_past_2_33_elements(canon):
    """More elements than 2^33, of which 16-byte accesses make few workgroups."""
    width, n = 8192, (1 << 20) + 5
    w = torch.randn(7, width, device="cuda").to(BF16)
    ids = torch.arange(n, device="cuda") % 8  # 7: outside the table
    got = canon.embedding(w, ids, scale=2.0)
    assert got.numel() > 1 << 33
    want = torch.cat([(w.float() * 2).to(BF16), torch.zeros(1, width, device="cuda").to(BF16)])
    for at in range(0, n, 1 << 17):
        assert torch.equal(got[at:at + (1 << 17)], want[ids[at:at + (1 << 17)]]), at


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("scale", [-1.0, float("inf"), float("-inf"), float("nan")])
def test_rows_outside_the_table_are_zero_for_any_scale(canon, dtype, scale):
    w = torch.ones(3, 9, dtype=dtype, device="cuda")
    ids = torch.tensor([-1, 1, 3, 2 ** 40], device="cuda")
    got = canon.embedding(w, ids, scale=scale)
    want = torch.zeros(4, 9, dtype=dtype)
    want[1] = scale
    assert torch.equal(torch.isnan(got).cpu(), torch.isnan(want))
    assert same_bits(torch.where(torch.isnan(got), 0, got), torch.where(torch.isnan(want), 0, want))


@pytest.mark.parametrize("tokens,rows,width,kernels", [
    (128, 1000, 4096, 1), (129, 1000, 4096, 1), (1024, 1000, 4096, 1), (1025, 1000, 4096, 3),
    (4096, 300, 4090, 3), (4096, 1000, 3580, 1), (4096, 1000, 3590, 3), (2000, 33000, 1000, 1),
    (2000, 34000, 1000, 3), (4097, 1000, 520, 3)])
def test_one_launch_only_where_it_gains(canon, tokens, rows, width, kernels):
    """Wide rows and large tables of more than 1024 tokens take three launches, whose
    time does not depend on how frequent an id is; the bits are the same."""
    dout = torch.randn(tokens, width, generator=torch.Generator().manual_seed(rows)).to(BF16)
    for kind in ("one", "zipf"):
        ids = make_ids(tokens, rows, kind, rows)
        d, i = dout.cuda(), ids.cuda()
        out = torch.full((rows, width), 7.0, dtype=BF16, device="cuda")
        assert launches(lambda: canon.embedding_grad(d, i, rows, out=out)) == kernels
        if rows <= 1000:
            assert same_bits(canon.embedding_grad(d, i, rows), grad_ref(dout, ids, rows, 1.0,
                                                                        dtype=BF16))
