"""fp64 oracle of the channels-last group norm with an activation, and its gradients.

TEST INFRASTRUCTURE ONLY.  It shares no code with the CUDA library.

x [N, S, C], G groups of neighbouring channels: xh = (x - mean) / sqrt(var + eps) over (S, C / G),
z = xh w + b, y = act(z), or z act(gate).  Pins: ``tests/test_group_norm_pins.py`` (central differences,
torch's group norm).
"""
from __future__ import annotations

import math

import numpy as np

_erf = np.vectorize(math.erf, otypes=[np.float64])


def _f64(a):
    if a is None:
        return None
    if hasattr(a, "detach"):
        return a.detach().to("cpu").double().numpy()
    return np.asarray(a, dtype=np.float64)


def act(name, z):
    """(act(z), act'(z))"""
    if name == "silu":
        s = 0.5 * (1 + np.tanh(0.5 * z))
        return z * s, s * (1 + z * (1 - s))
    if name == "gelu":
        c = 0.5 * (1 + _erf(z / math.sqrt(2)))
        return z * c, c + z * np.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    return z, np.ones_like(z)


def _norm(x, G, eps):
    N, S, C = x.shape
    g = x.reshape(N, S, G, C // G)
    mean = g.mean(axis=(1, 3))
    var = ((g - mean[:, None, :, None]) ** 2).mean(axis=(1, 3))
    rstd = 1 / np.sqrt(var + eps)
    xh = ((g - mean[:, None, :, None]) * rstd[:, None, :, None]).reshape(N, S, C)
    return xh, mean, rstd


def group_norm_ref(x, G, weight=None, bias=None, gate=None, eps=1e-5, activation="none"):
    """x [N, S, C].  Returns (y, mean, rstd) in fp64."""
    x, weight, bias, gate = map(_f64, (x, weight, bias, gate))
    xh, mean, rstd = _norm(x, G, eps)
    z = xh * (1 if weight is None else weight) + (0 if bias is None else bias)
    y = act(activation, z)[0] if gate is None else z * act(activation, gate)[0]
    return y, mean, rstd


def group_norm_grad_ref(x, G, weight=None, bias=None, gate=None, eps=1e-5, activation="none", *, dy):
    """Returns a dict of fp64 gradients: dx, dweight, dbias, and dgate with a gate."""
    x, weight, bias, gate, dy = map(_f64, (x, weight, bias, gate, dy))
    N, S, C = x.shape
    xh, mean, rstd = _norm(x, G, eps)
    w = np.ones(C) if weight is None else weight
    z = xh * w + (0 if bias is None else bias)
    out = {}
    if gate is None:
        dz = dy * act(activation, z)[1]
    else:
        value, slope = act(activation, gate)
        dz = dy * value
        out["dgate"] = dy * z * slope
    out["dweight"], out["dbias"] = (dz * xh).sum((0, 1)), dz.sum((0, 1))
    dn = (dz * w).reshape(N, S, G, -1)
    g = xh.reshape(N, S, G, -1)
    dx = dn - dn.mean((1, 3), keepdims=True) - g * (dn * g).mean((1, 3), keepdims=True)
    out["dx"] = (dx * rstd[:, None, :, None]).reshape(N, S, C)
    return out
