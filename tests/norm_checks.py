"""Reference and tolerances of the group norm's gradients, term by term.

The backward pass takes the forward's fp32 mean and rstd as inputs, so the reference here takes the same values: what
they lack of the exact statistics is no error of the gradient, and nothing below grows with |x|max rstd.  With
u = 2^-24, an error bound of each value (E of it) in the order of the computation:

    xh = (x - mean) rstd            2 u |xh|
    z  = xh w + b                   |w| E(xh) + u |z|
    act(t), act'(t)                 2^-20 (1 + |t|); exact without an activation.  |act''| <= 0.8 (SiLU 0.5, GELU 2 phi(0))
    dz = dy act'(z)                 |dy| (E(act') + 0.8 E(z)) + u |dz|;   with a gate  |dy| E(act(gate)) + u |dz|
    dgate = dy z act'(gate)         |dy| (|act'| E(z) + |z| E(act')) + 2 u |dgate|
    dn = dz w                       |w| E(dz) + u |dn|
    m1 = mean dn, m2 = mean dn xh   the mean of the terms' errors (E(dn);  |xh| E(dn) + 3 u |dn xh|) and K u of the mean
                                    of the terms' absolute values, K the additions that a term passes
    dx = rstd (dn - m1 - xh m2)     rstd (E(dn) + E(m1) + |xh| E(m2) + 3 u (|dn| + |m1| + |xh m2|)) + 2 u |dx|
    dweight, dbias                  sum of the terms' errors and K u of the sum of their absolute values

and 2^-8 of the value where it is rounded to bf16.  K: a thread's positions, S / RL with RL = 256 / (vectors of a position)
row lanes, then at most 300 + D over row lanes, channels, lanes and tiles; for a channel's sums at most N S + 300.
"""
import math

import torch

U = 2.0 ** -24


def activation_of(name, t):
    """act(t), act'(t)"""
    if name == "silu":
        s = torch.sigmoid(t)
        return t * s, s * (1 + t * (1 - s))
    if name == "gelu":
        c = 0.5 * (1 + torch.erf(t * math.sqrt(0.5)))
        return t * c, c + t * torch.exp(-0.5 * t * t) / math.sqrt(2 * math.pi)
    return t, torch.ones_like(t)


def grad_reference(x, G, mean, rstd, weight=None, bias=None, gate=None, *, dy, activation="none"):
    """x, gate, dy [N, S, C] with the statistics mean, rstd [N, G].  Returns (gradients, tolerances), dicts of fp64."""
    N, S, C = x.shape
    D = C // G
    bf16 = x.dtype == torch.bfloat16
    rounded = 2.0 ** -8 if bf16 else 0.0
    vector = 16 // x.element_size() if C % (16 // x.element_size()) == 0 else 1
    K = S / max(1, 256 // (C // vector)) + 300 + D

    def wide(t):
        return t.double().view(N, 1, G, 1)

    def means(t):
        return t.mean(dim=(1, 3), keepdim=True)

    def groups(t):
        return t.double().view(N, S, G, D)

    mean, rstd, x, dy = wide(mean), wide(rstd), groups(x), groups(dy)
    w = torch.ones((), dtype=torch.float64, device=x.device) if weight is None else weight.double().view(G, D)
    b = 0.0 if bias is None else bias.double().view(G, D)
    act_err = 0.0 if activation == "none" else 2.0 ** -20
    curve = 0.0 if activation == "none" else 0.8
    xh = (x - mean) * rstd
    z = xh * w + b
    e_z = 2 * U * (xh * w).abs() + U * z.abs()
    grads, tols = {}, {}
    if gate is None:
        slope = activation_of(activation, z)[1]
        dz = dy * slope
        e_dz = dy.abs() * (act_err * (1 + z.abs()) + curve * e_z) + U * dz.abs()
    else:
        t = groups(gate)
        value, slope = activation_of(activation, t)
        dz = dy * value
        e_t = act_err * (1 + t.abs())
        e_dz = dy.abs() * e_t + U * dz.abs()
        dgate = dy * z * slope
        grads["dgate"] = dgate.reshape(N, S, C)
        tols["dgate"] = (dy.abs() * (slope.abs() * e_z + z.abs() * e_t) + (2 * U + rounded) * dgate.abs()).reshape(N, S, C)
    dn = dz * w
    e_dn = w.abs() * e_dz + U * dn.abs()
    m1, m2 = means(dn), means(dn * xh)
    e_m1 = means(e_dn) + K * U * means(dn.abs())
    e_m2 = means(xh.abs() * e_dn) + (K + 3) * U * means((dn * xh).abs())
    dx = rstd * (dn - m1 - xh * m2)
    e_dx = rstd * (e_dn + e_m1 + xh.abs() * e_m2 + 3 * U * (dn.abs() + m1.abs() + (xh * m2).abs()))
    grads["dx"], tols["dx"] = dx.reshape(N, S, C), (e_dx + (2 * U + rounded) * dx.abs()).reshape(N, S, C)
    k = (N * S + 300) * U
    if weight is not None:
        grads["dweight"] = (dz * xh).sum((0, 1)).reshape(C)
        tols["dweight"] = (e_dz * xh.abs() + (3 * U + k) * (dz * xh).abs()).sum((0, 1)).reshape(C)
    if bias is not None:
        grads["dbias"] = dz.sum((0, 1)).reshape(C)
        tols["dbias"] = (e_dz + k * dz.abs()).sum((0, 1)).reshape(C)
    return grads, tols


def wrong(got, ref, tol):
    """How many elements are out of tolerance (or not numbers), and the worst one's multiple of it."""
    err = (got.double() - ref).abs()
    off = ~(err <= tol + 1e-30)
    return int(off.sum()), float((err / (tol + 1e-30)).max())


def check_grads(got, x, G, mean, rstd, weight=None, bias=None, gate=None, *, dy, activation="none"):
    grads, tols = grad_reference(x, G, mean, rstd, weight, bias, gate, dy=dy, activation=activation)
    assert set(got) == set(grads)
    for name in grads:
        n, worst = wrong(got[name], grads[name], tols[name])
        assert n == 0, f"{name}: {n} of {grads[name].numel()} off, worst {worst:.3g} of the tolerance"
