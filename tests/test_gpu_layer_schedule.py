"""The norm's kernels walk their rows with any number of workgroups: the same bits."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def canon():
    import scan_canonical_reduce_amd as c
    yield c
    c.set_schedule("grid", 0)


@pytest.fixture(autouse=True)
def seed():
    torch.manual_seed(5)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,width", [(131, 40), (37, 1000), (11, 4096), (9, 9000), (7, 20001)])
def test_norm_grid(canon, dtype, rows, width):
    g = torch.Generator().manual_seed(width)
    x, r, dout = (torch.randn(rows, width, generator=g).to(dtype).cuda() for _ in range(3))
    w = torch.rand(width, generator=g).cuda()

    def both():
        stats = canon.layer_norm_stats(x)
        out, total = canon.add_layer_norm(x, r, w, w, stats=stats)
        alone = canon.layer_norm(x, w)
        a, b = x.clone(), r.clone()  # in place
        canon.add_layer_norm(a, b, w, w, sum_out=a, out=b)
        grads = canon.layer_norm_grad(dout, total, w, stats, w, dsum=r)
        return [out, total, stats, alone, a, b, *grads]

    want = both()
    assert torch.equal(want[4], want[1]) and torch.equal(want[5], want[0])
    for grid in (1, 3, 5):
        with canon.schedule(grid=grid):
            for got, one in zip(both(), want):
                assert torch.equal(got, one), grid


def test_the_cap_is_obeyed(canon):
    """One workgroup takes many times as long as hundreds."""
    w = torch.ones(20001, device="cuda")

    def least(call):
        times = []
        for _ in range(4):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            call()
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    for width in (1024, 20001):
        x = torch.randn(2048, width, device="cuda")
        stats = canon.layer_norm_stats(x)
        out = canon.layer_norm(x, w[:width], stats=stats)
        calls = [lambda: canon.layer_norm(x, w[:width], out=out)]
        if width > 8192:  # dx has a kernel of its own
            calls.append(lambda: canon.layer_norm_grad(out, x, w[:width], stats, dx=out))
        for call in calls:
            free = least(call)
            with canon.schedule(grid=1):
                assert least(call) > 4 * free
