"""The float64 formulas that GPU tests compare with, against autograd (CPU)."""
import pytest

torch = pytest.importorskip("torch")

import seq_ref  # noqa: E402


@pytest.mark.parametrize("groups,states", [(1, 16), (2, 5)])
def test_scan_grads(groups, states):
    n, rows, ch = 3, 11, 12
    g = torch.Generator().manual_seed(states)

    def normal(*s):
        return torch.randn(*s, generator=g, dtype=torch.float64)

    d = dict(u=normal(n, rows, ch), delta=normal(n, rows, ch), z=normal(n, rows, ch),
             dout=normal(n, rows, ch), B=normal(n, rows, groups, states),
             C=normal(n, rows, groups, states), A=-torch.exp(normal(ch, states)), D=normal(ch),
             bias=normal(ch), init=normal(n, ch, states), dfinal=normal(n, ch, states))
    names = ["u", "delta", "A", "B", "C", "D", "z", "bias", "init"]
    e = {k: v.clone().requires_grad_(k in names) for k, v in d.items()}
    outs, finals = zip(*(seq_ref.scan_one(e["u"][i], e["delta"][i], e["A"], e["B"][i], e["C"][i],
                                          e["D"], e["z"][i], e["bias"], True, e["init"][i])
                         for i in range(n)))
    loss = (torch.stack(outs) * d["dout"]).sum() + (torch.stack(finals) * d["dfinal"]).sum()
    want = torch.autograd.grad(loss, [e[k] for k in names])
    out, final, got = seq_ref.scan_grads(d)
    assert torch.allclose(out, torch.stack(outs).detach(), rtol=1e-12, atol=1e-12)
    assert torch.allclose(final, torch.stack(finals).detach(), rtol=1e-12, atol=1e-12)
    _, _, size = seq_ref.scan_grads(d, absolute=True)
    for k, w in zip(names, want):
        assert torch.allclose(got[k], w, rtol=1e-11, atol=1e-11), k
        assert (size[k] >= got[k].abs() - 1e-12).all(), k
