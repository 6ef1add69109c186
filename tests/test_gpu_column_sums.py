"""Parameter gradients' sums over rows: 16 lanes in row order, then the pairwise tree,
bit for bit at every number of rows around a lane's steps."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def canon():
    import scan_canonical_reduce_amd as c
    return c


def by_lanes(parts):
    """float32 sums of the rows of parts"""
    lanes = [np.zeros(parts.shape[1], np.float32) for _ in range(16)]
    for r, row in enumerate(parts):
        lanes[r % 16] = lanes[r % 16] + row
    d = 1
    while d < 16:
        for i in range(0, 16, 2 * d):
            lanes[i] = lanes[i] + lanes[i + d]
        d *= 2
    return lanes[0]


@pytest.mark.parametrize("width", [70, 300])
def test_every_number_of_rows(canon, width):
    """Up to 512 rows a norm's bias gradient has a part for each row: the row itself."""
    g = torch.Generator().manual_seed(width)
    x = torch.randn(512, width, generator=g).cuda()
    dout = torch.randn(512, width, generator=g) * 10.0 ** torch.randint(-3, 4, (512, 1), generator=g)
    w = torch.ones(width, device="cuda")
    for rows in list(range(1, 145)) + [255, 256, 257, 500, 501, 511, 512]:
        stats = canon.layer_norm_stats(x[:rows])
        canon.layer_norm(x[:rows], w, w, stats=stats)
        got = canon.layer_norm_grad(dout[:rows].cuda(), x[:rows], w, stats, w).dbias.cpu().numpy()
        assert got.tobytes() == by_lanes(dout[:rows].numpy()).tobytes(), rows
