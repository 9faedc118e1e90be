"""fp64 oracle of the decay scan (linear attention with one fixed decay per head) and its gradients.

TEST INFRASTRUCTURE ONLY.  It shares no code with the CUDA library.

    S_t = a_h S_{t-1} + v_t k_t^T,   o_t = S_t q_t

one token at a time, all (b, h) at once; query head h reads key / value head h // (H / Hkv); tokens
t >= lengths[b] are skipped and their outputs are zero.  Gradients, with G_t that of S_t:

    G_t += do_t q_t^T;  dq_t = S_t^T do_t;  dk_t = G_t^T v_t;  dv_t = G_t k_t;  G_{t-1} = a_h G_t;  dS0 = G_0

Pins: ``tests/test_decay_pins.py`` (central differences of the forward; the delta-rule oracle with the
erase gate at zero).
"""
from __future__ import annotations

import numpy as np


def _f64(a):
    if a is None:
        return None
    if hasattr(a, "detach"):
        return a.detach().to("cpu").double().numpy()
    return np.asarray(a, dtype=np.float64)


def _setup(q, k, v, decay, S0, lengths):
    q, k, v, decay, S0 = map(_f64, (q, k, v, decay, S0))
    B, T, H, dk = q.shape
    rep = H // k.shape[2]
    k, v = np.repeat(k, rep, axis=2), np.repeat(v, rep, axis=2)
    n = np.full(B, T) if lengths is None else np.clip(np.asarray(_f64(lengths)).astype(np.int64), 0, T)
    live = np.arange(T)[None] < n[:, None]  # [B, T]
    for x in (q, k, v):
        x[~live] = 0.0
    S = np.zeros((B, H, v.shape[-1], dk)) if S0 is None else S0.copy()
    return q, k, v, decay, S, live, rep


def decay_scan_ref(q, k, v, decay, S0=None, lengths=None):
    """Returns (o [B,T,H,dv], S_final [B,H,dv,dk]) in fp64."""
    q, k, v, a, S, live, _ = _setup(q, k, v, decay, S0, lengths)
    B, T, H, _ = q.shape
    o = np.zeros((B, T, H, v.shape[-1]))
    for t in range(T):
        new = a[None, :, None, None] * S + v[:, t, :, :, None] * k[:, t, :, None, :]
        m = live[:, t][:, None, None, None]
        S = np.where(m, new, S)
        o[:, t] = np.where(m[..., 0], np.einsum("bhvk,bhk->bhv", S, q[:, t]), 0.0)
    return o, S


def decay_scan_grad_ref(q, k, v, decay, S0=None, lengths=None, *, do, dS_final=None):
    """Returns a dict of fp64 gradients dq, dk, dv (shapes of q, k, v) and dS0."""
    kv_heads = k.shape[2]
    do, dS = _f64(do), _f64(dS_final)
    q, k, v, a, S, live, rep = _setup(q, k, v, decay, S0, lengths)
    B, T, H, _ = q.shape
    do = np.where(live[:, :, None, None], do, 0.0)
    states = []
    for t in range(T):
        m = live[:, t][:, None, None, None]
        S = np.where(m, a[None, :, None, None] * S + v[:, t, :, :, None] * k[:, t, :, None, :], S)
        states.append(S)
    G = np.zeros_like(S) if dS is None else dS.copy()
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for t in reversed(range(T)):
        m = live[:, t][:, None, None, None]
        G = G + do[:, t, :, :, None] * q[:, t, :, None, :]
        dq[:, t] = np.einsum("bhvk,bhv->bhk", states[t], do[:, t])
        dk[:, t] = np.where(m[..., 0], np.einsum("bhvk,bhv->bhk", G, v[:, t]), 0.0)
        dv[:, t] = np.where(m[..., 0], np.einsum("bhvk,bhk->bhv", G, k[:, t]), 0.0)
        G = np.where(m, a[None, :, None, None] * G, G)
    fold = lambda x: x.reshape(B, T, kv_heads, rep, -1).sum(3)  # noqa: E731
    return {"dq": dq, "dk": fold(dk), "dv": fold(dv), "dS0": G}
