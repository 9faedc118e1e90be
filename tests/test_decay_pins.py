"""Pins of the decay scan's oracle (CPU): the delta-rule oracle with no erase, closed forms, central
differences of the forward."""
import numpy as np
import pytest
import torch

import oracle
from oracle.decay_scan import decay_scan_grad_ref, decay_scan_ref


def draw(seed, B=2, T=9, H=4, Hkv=2, dk=5, dv=3):
    r = np.random.RandomState(seed)
    return (r.randn(B, T, H, dk), r.randn(B, T, Hkv, dk), r.randn(B, T, Hkv, dv), np.array([0.0, 0.5, 0.9, 1.0])[:H],
            r.randn(B, H, dv, dk))


def test_equals_the_delta_rule_without_erase():
    g = torch.Generator().manual_seed(0)
    B, T, H, d = 2, 40, 3, 32
    q, k, v = (torch.randn(B, T, H, d, generator=g) for _ in range(3))
    a = torch.tensor([0.3, 0.9, 1.0])
    alpha = a.expand(B, T, H).contiguous()
    zero = torch.zeros(B, T, H)
    o, S = oracle.scan_ref(q=q, k=k, v=None, alpha=alpha, beta=zero, u=v[:, :, :, None].contiguous(),
                           w=k[:, :, :, None].contiguous(), S0=None)
    o2, S2 = decay_scan_ref(q, k, v, a)
    np.testing.assert_allclose(o2, o, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(S2, S, rtol=1e-12, atol=1e-12)


def test_quadratic_form_and_shared_heads():
    q, k, v, a, S0 = draw(1)
    o, S = decay_scan_ref(q, k, v, a, S0)
    T = q.shape[1]
    gap = np.arange(T)[:, None] - np.arange(T)
    for b in range(2):
        for h in range(4):
            M = np.where(gap >= 0, a[h] ** np.maximum(gap, 0), 0.0)
            ref = (M * (q[b, :, h] @ k[b, :, h // 2].T)) @ v[b, :, h // 2]
            ref += (a[h] ** (np.arange(T) + 1))[:, None] * (q[b, :, h] @ S0[b, h].T)
            np.testing.assert_allclose(o[b, :, h], ref, rtol=1e-12, atol=1e-12)


def test_padding_is_no_part_of_the_sequence():
    q, k, v, a, S0 = draw(2)
    n = np.array([4, 0])
    k[0, 4:], v[1] = np.nan, np.nan
    o, S = decay_scan_ref(q, k, v, a, S0, n)
    o1, S1 = decay_scan_ref(q[:1, :4], k[:1, :4], v[:1, :4], a, S0[:1])
    np.testing.assert_array_equal(o[:1, :4], o1)
    np.testing.assert_array_equal(S[:1], S1)
    assert (o[0, 4:] == 0).all() and (o[1] == 0).all() and (S[1] == S0[1]).all()


@pytest.mark.parametrize("lengths", [None, np.array([9, 5])])
def test_gradients_by_central_differences(lengths):
    q, k, v, a, S0 = draw(3)
    r = np.random.RandomState(4)
    do, dS = r.randn(2, 9, 4, 3), r.randn(2, 4, 3, 5)

    def loss(q, k, v, S0):
        o, S = decay_scan_ref(q, k, v, a, S0, lengths)
        return (o * do).sum() + (S * dS).sum()

    got = decay_scan_grad_ref(q, k, v, a, S0, lengths, do=do, dS_final=dS)
    x = {"dq": q, "dk": k, "dv": v, "dS0": S0}
    for name, t in x.items():
        for _ in range(25):
            i = tuple(r.randint(n) for n in t.shape)
            args = {n: u.copy() for n, u in x.items()}
            e = 1e-5
            args[name][i] += e
            up = loss(*args.values())
            args[name][i] -= 2 * e
            down = loss(*args.values())
            # the loss is at most quadratic in one input: differences are exact up to rounding,
            # about 2^-53 |loss| / e
            assert abs((up - down) / (2 * e) - got[name][i]) < 1e-8, (name, i)
