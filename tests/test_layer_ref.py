"""The float64 forms that the GPU tests of the layer operators compare with, against
autograd and differences (no GPU)."""
import pytest

torch = pytest.importorskip("torch")

import layer_ref  # noqa: E402


def normal(*shape, seed=[0]):
    seed[0] += 1
    return torch.randn(*shape, dtype=torch.float64, generator=torch.Generator().manual_seed(seed[0]))


def differences(loss, leaves, grads):
    """Directional derivatives by central differences."""
    for k in leaves:
        v, h = normal(*leaves[k].shape), 1e-6
        up, down = (loss(dict(leaves, **{k: leaves[k] + s * h * v})) for s in (1, -1))
        want = float(up - down) / (2 * h)
        assert abs(float((grads[k] * v).sum()) - want) <= 1e-6 * (1 + abs(want)), k


def test_norm_gradient():
    x, w, dout, dsum = normal(5, 17), normal(17), normal(5, 17), normal(5, 17)
    (dx, _), (dw, _), (db, _) = layer_ref.norm_grad(dout, x, w, dsum, 1e-5)
    leaves = dict(x=x, w=w, b=normal(17))

    def loss(p):
        out = layer_ref.norm(p["x"], p["w"], p["b"], 1e-5)[0]
        return (out * dout).sum() + (p["x"] * dsum).sum()

    differences(loss, leaves, dict(x=dx, w=dw, b=db))


@pytest.mark.parametrize("decay", [False, True])
@pytest.mark.parametrize("gated", [False, True])
def test_recurrence_gradient(decay, gated):
    leaves = dict(x=normal(2, 9, 4), gate=normal(2, 9, 4), init=normal(2, 4))
    if gated:
        leaves["input_gate"] = normal(2, 9, 4)
    if decay:
        leaves["decay"] = normal(4).exp()
    dout, dfinal = normal(2, 9, 4), normal(2, 4)
    got = layer_ref.recur(**leaves, dout=dout, dfinal=dfinal)

    def loss(p):
        r = layer_ref.recur(**p)
        return (r["out"][0] * dout).sum() + (r["final"][0] * dfinal).sum()

    differences(loss, leaves, {k: got[k][0] for k in leaves})
    # and by autograd of the recurrence written out
    e = {k: v.clone().requires_grad_() for k, v in leaves.items()}
    r = torch.sigmoid(e["gate"])
    a = torch.exp(-e["decay"] * r) if decay else r
    c = torch.sqrt(1 - a * a) if decay else 1 - a
    v = c * e["x"] * (torch.sigmoid(e["input_gate"]) if gated else 1)
    h, total = e["init"], 0
    for t in range(9):
        h = a[:, t] * h + v[:, t]
        total = total + (h * dout[:, t]).sum()
    want = torch.autograd.grad(total + (h * dfinal).sum(), list(e.values()))
    for k, g in zip(e, want):
        assert torch.allclose(got[k][0], g, rtol=1e-10, atol=1e-12), k
