"""The gradient check of tests/norm_checks.py on CPU: its reference is the oracle's formula, a plain computation in 32 bits
passes it, and a gradient that lacks one of its terms does not."""
import numpy as np
import pytest
import torch

from oracle.group_norm import group_norm_grad_ref
from tests.norm_checks import activation_of, check_grads, grad_reference, wrong

BF, F32 = torch.bfloat16, torch.float32
SHAPES = [(4, 1, 64, 2), (4, 300, 64, 2), (1, 5000, 8, 2), (5, 1, 640, 5), (3, 50, 96, 8), (2, 40, 30, 5)]


def make(seed, N, S, C, io, mean, std):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return {"x": (mean + std * r(N, S, C)).to(io), "dy": r(N, S, C).to(io), "gate": r(N, S, C).to(io),
            "weight": 1 + 0.3 * r(C), "bias": 0.3 * r(C)}


def statistics(x, G, eps=1e-5):
    g = x.double().view(x.shape[0], x.shape[1], G, -1)
    var, mean = torch.var_mean(g, dim=(1, 3), unbiased=False)
    return mean.float(), (var + eps).rsqrt().float()


def plain(x, G, mean, rstd, weight, bias, gate, dy, activation, without=()):
    """The gradients in 32 bits, without some of dx's terms."""
    N, S, C = x.shape
    io = x.dtype
    xh = ((x.float().view(N, S, G, -1) - mean.view(N, 1, G, 1)) * rstd.view(N, 1, G, 1)).view(N, S, C)
    z = xh if weight is None else xh * weight + bias
    out = {}
    if gate is None:
        dz = dy.float() * activation_of(activation, z)[1]
    else:
        value, slope = activation_of(activation, gate.float())
        dz = dy.float() * value
        out["dgate"] = (dy.float() * z * slope).to(io)
    if weight is not None:
        out["dweight"], out["dbias"] = (dz * xh).sum((0, 1)), dz.sum((0, 1))
    dn = (dz if weight is None else dz * weight).view(N, S, G, -1)
    n = xh.view(N, S, G, -1)
    m1 = 0 if "m1" in without else dn.mean((1, 3), keepdim=True)
    m2 = 0 if "m2" in without else (dn * n).mean((1, 3), keepdim=True)
    out["dx"] = ((dn - m1 - n * m2) * rstd.view(N, 1, G, 1)).view(N, S, C).to(io)
    return out


@pytest.mark.parametrize("activation", ["none", "silu", "gelu"])
@pytest.mark.parametrize("gated", [False, True])
def test_the_reference_is_the_oracles(activation, gated):
    x = {n: t.double() for n, t in make(1, 3, 5, 12, F32, 0.3, 1.0).items()}
    gate = x["gate"] if gated else None
    g = x["x"].view(3, 5, 4, 3)
    var, mean = torch.var_mean(g, dim=(1, 3), unbiased=False)
    got, _ = grad_reference(x["x"], 4, mean, (var + 1e-5).rsqrt(), x["weight"], x["bias"], gate, dy=x["dy"], activation=activation)
    ref = group_norm_grad_ref(x["x"], 4, x["weight"], x["bias"], gate, activation=activation, dy=x["dy"])
    for n in got:
        np.testing.assert_allclose(got[n].numpy(), ref[n], rtol=1e-11, atol=1e-12)


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("mean,std", [(0.3, 1.0), (1000.0, 0.5)])
@pytest.mark.parametrize("activation,gated,affine", [("none", False, True), ("silu", True, True), ("gelu", False, False)])
@pytest.mark.parametrize("N,S,C,G", SHAPES)
def test_right_passes_and_wrong_does_not(io, mean, std, activation, gated, affine, N, S, C, G):
    x = make(2, N, S, C, io, mean, max(std, 4.0) if io == BF and mean > 100 else std)  # (bf16 steps by 4 at 1000)
    m, r = statistics(x["x"], G)
    args = (x["x"], G, m, r, x["weight"] if affine else None, x["bias"] if affine else None, x["gate"] if gated else None)
    kw = {"dy": x["dy"], "activation": activation}
    check_grads(plain(*args, **kw), *args, **kw)
    grads, tols = grad_reference(*args, **kw)
    for without in (("m1",), ("m2",), ("m1", "m2")):
        dx = plain(*args, **kw, without=without)["dx"]
        assert wrong(dx, grads["dx"], tols["dx"])[0] > 0, without
    dx = plain(*args, **kw)["dx"]
    assert wrong(torch.zeros_like(dx), grads["dx"], tols["dx"])[0] > 0.9 * dx.numel()
    assert wrong(100 * dx, grads["dx"], tols["dx"])[0] > 0.9 * dx.numel()
    # an offset of 2^-11 (bf16: 2^-5) of the largest: K U is below 2^-13 for these shapes, a rounding to bf16 2^-8
    assert wrong(dx.double() + 2.0 ** (-5 if io == BF else -11) * dx.abs().max(), grads["dx"], tols["dx"])[0] > 0
