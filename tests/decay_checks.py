"""Inputs and tolerances of the decay scan's GPU tests.

Every output is a sum  sum_j a^(i-j) (x_i . y_j) z_j + a^(i+1) R x_i  (the module comment of decay.cuh).
M below is the same sum over absolute values, which the oracle gives for absolute inputs.

bf16 outputs: the result is rounded once (at most 2^-8 |o|), and inside, each chunk product a^(i-j) (x_i . y_j)
and each state element is rounded once where it enters the output's product (at most 2^-8 M together, each
term having exactly one of the two).  Norm-wise, with independent roundings of terms that do not cancel
systematically (random inputs), each of the two is at most 2^-8 of the output's norm: together below 2 x 2^-8.
fp32 results (outputs with fp32 inputs, states always): at most K = 2 x 128 + 64 + T / 64 additions and
multiplications of relative error 2^-24 on the way of any term: K 2^-24 M, below 2^-14 M for T < 45000.
Norm-wise the errors add up like a random walk: sqrt(K) 2^-24, below 2^-18 for K < 4096.
"""
import numpy as np
import torch

from oracle.decay_scan import decay_scan_grad_ref, decay_scan_ref


def make(seed, B, T, H, Hkv, dk, dv, io=torch.bfloat16, S0=True, ragged=False, decay=None, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    x = {"q": torch.randn(B, T, H, dk, generator=g).to(io),
         "k": torch.nn.functional.normalize(torch.randn(B, T, Hkv, dk, generator=g), dim=-1).to(io),
         "v": torch.randn(B, T, Hkv, dv, generator=g).to(io),
         "decay": torch.tensor((decay or [0.9, 1.0, 0.0, 0.999, 0.3, 1 - 2.0 ** -12, 1e-3, 0.97] * 4)[:H]),
         "S0": 0.3 * torch.randn(B, H, dv, dk, generator=g) if S0 else None,
         "lengths": None}
    if ragged:
        n = torch.randint(0, T + 1, (B,), generator=g, dtype=torch.int32)
        n[0] = T
        x["lengths"] = n
    return {n: None if t is None else t.to(device) for n, t in x.items()}


def _abs(t):
    return None if t is None else torch.nan_to_num(t.float()).abs()


def _np(t):
    return t.detach().double().cpu().numpy()


def check(name, got, ref, mass, bf16, random=True):
    got = _np(got)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert np.isfinite(got).all(), f"{name}: not finite"
    err = np.abs(got - ref)
    tol = (2.0 ** -8 * (np.abs(ref) + mass) if bf16 else 2.0 ** -14 * mass) + 1e-30
    assert (err <= tol).all(), f"{name}: {(err > tol).sum()} of {err.size} off, worst {(err / tol).max():.3g} of the tolerance"
    if random:
        norm = np.linalg.norm(ref)
        lim = (2.0 ** -7 if bf16 else 2.0 ** -18) * norm
        assert np.linalg.norm(err) <= lim + 1e-30, f"{name}: error norm {np.linalg.norm(err) / (norm + 1e-300):.3g}"


def check_fwd(x, o, S, random=True):
    bf16 = x["q"].dtype == torch.bfloat16
    ref = decay_scan_ref(**x)
    mass = decay_scan_ref(**{n: t if n in ("decay", "lengths") else _abs(t) for n, t in x.items()})
    check("o", o, ref[0], mass[0], bf16, random)
    if S is not None:
        check("S_final", S, ref[1], mass[1], False, random)


def check_bwd(x, dO, dS, got, random=True):
    bf16 = x["q"].dtype == torch.bfloat16
    ref = decay_scan_grad_ref(**x, do=dO, dS_final=dS)
    mass = decay_scan_grad_ref(**{n: t if n in ("decay", "lengths") else _abs(t) for n, t in x.items()}, do=_abs(dO),
                               dS_final=_abs(dS))
    for name in ("dq", "dk", "dv", "dS0"):
        if got[name] is not None:
            check(name, got[name], ref[name], mass[name], bf16 and name != "dS0", random)
