"""Pins of the group norm's oracle (CPU): torch's group norm and its autograd in 64 bits, central
differences."""
import numpy as np
import pytest
import torch

from oracle.group_norm import group_norm_grad_ref, group_norm_ref

F = torch.nn.functional
ACT = {"none": lambda u: u, "silu": F.silu, "gelu": F.gelu}


@pytest.mark.parametrize("activation", ["none", "silu", "gelu"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("S", [1, 5])
def test_matches_torch(activation, gated, S):
    g = torch.Generator().manual_seed(1)
    N, C, G = 3, 12, 4
    x, gate, dy = (torch.randn(N, S, C, generator=g, dtype=torch.float64) for _ in range(3))
    w, b = (torch.randn(C, generator=g, dtype=torch.float64) for _ in range(2))
    leaves = [t.requires_grad_(True) for t in (x, w, b, gate)]
    z = F.group_norm(x.transpose(1, 2), G, w, b, 1e-3).transpose(1, 2)
    y = z * ACT[activation](gate) if gated else ACT[activation](z)
    y.backward(dy)
    args = (x.detach(), G, w.detach(), b.detach(), gate.detach() if gated else None)
    got, _, _ = group_norm_ref(*args, eps=1e-3, activation=activation)
    np.testing.assert_allclose(got, y.detach().numpy(), rtol=1e-12, atol=1e-12)
    grads = group_norm_grad_ref(*args, eps=1e-3, activation=activation, dy=dy)
    for name, leaf in zip(("dx", "dweight", "dbias", "dgate"), leaves):
        if name in grads:
            np.testing.assert_allclose(grads[name], leaf.grad.numpy(), rtol=1e-11, atol=1e-11)


def test_gradient_by_central_differences():
    r = np.random.RandomState(0)
    x, dy, gate, w, b = r.randn(2, 3, 8), r.randn(2, 3, 8), r.randn(2, 3, 8), r.randn(8), r.randn(8)
    grads = group_norm_grad_ref(x, 2, w, b, gate, activation="silu", dy=dy)
    e = 1e-5
    for _ in range(30):
        i = tuple(r.randint(n) for n in x.shape)
        for name, t in (("dx", x), ("dgate", gate)):
            t[i] += e
            up = (group_norm_ref(x, 2, w, b, gate, activation="silu")[0] * dy).sum()
            t[i] -= 2 * e
            down = (group_norm_ref(x, 2, w, b, gate, activation="silu")[0] * dy).sum()
            t[i] += e
            assert abs((up - down) / (2 * e) - grads[name][i]) < 1e-7
