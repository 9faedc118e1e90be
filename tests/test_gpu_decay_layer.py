"""The decay scan and the group norm together, as a layer runs them: a prompt, its gradients, single
tokens behind it, and chunk-by-chunk streaming with the output norm."""
import numpy as np
import pytest
import torch

from oracle.decay_scan import decay_scan_grad_ref, decay_scan_ref
from oracle.group_norm import group_norm_grad_ref, group_norm_ref
from tests.decay_checks import make

pytestmark = pytest.mark.gpu


def prism():
    from delta_rule_sequence_b200 import prism as P

    return P


def layer_inputs(seed, B, T, H, Hkv, d):
    x = make(seed, B, T, H, Hkv, d, d, ragged=B > 1, decay=[0.5, 0.9, 0.99, 0.999])
    g = torch.Generator().manual_seed(seed + 1)
    x["gate"] = torch.randn(B * T, H * d, generator=g).bfloat16().cuda()
    x["weight"] = (1 + 0.2 * torch.randn(H * d, generator=g)).cuda()
    x["dy"] = torch.randn(B * T, H * d, generator=g).bfloat16().cuda()
    return x


def test_prompt_then_gradients_then_single_tokens():
    P = prism()
    B, T, H, Hkv, d = 3, 310, 4, 2, 64
    x = layer_inputs(1, B, T, H, Hkv, d)
    q, k, v, a, S0, n = (x[i] for i in ("q", "k", "v", "decay", "S0", "lengths"))
    o, S = P.prism_decay_scan_fwd(q, k, v, a, S0, n)
    flat = o.view(B * T, H * d)
    y, mean, rstd = P.prism_group_norm_fwd(flat, H, x["weight"], None, x["gate"], activation="silu")
    g = P.prism_group_norm_bwd(flat, H, mean, rstd, x["weight"], None, x["gate"], dy=x["dy"], activation="silu")
    gs = P.prism_decay_scan_bwd(q, k, v, a, S0, n, dO=g["dx"].view(B, T, H, d))
    one = {i: torch.randn(B, 1, h, d, device="cuda").bfloat16() for i, h in (("q", H), ("k", Hkv), ("v", Hkv))}
    state = S.clone()
    o1 = P.prism_decay_step(one["q"], one["k"], one["v"], a, state)
    torch.cuda.synchronize()

    # each stage against its oracle on the values that it was given, norm-wise: the result's rounding and
    # one inner rounding of at most 2^-8 each
    def close(name, got, ref, lim=2.0 ** -7):
        e = np.linalg.norm(got.double().cpu().numpy().reshape(ref.shape) - ref) / np.linalg.norm(ref)
        assert e < lim, (name, e)

    o_ref, S_ref = decay_scan_ref(q, k, v, a, S0, n)
    close("o", o, o_ref)
    close("S", S, S_ref, 2.0 ** -18)
    y_ref, _, _ = group_norm_ref(flat[:, None], H, x["weight"], None, x["gate"][:, None], activation="silu")
    close("y", y, y_ref)
    g_ref = group_norm_grad_ref(flat[:, None], H, x["weight"], None, x["gate"][:, None], activation="silu", dy=x["dy"][:, None])
    live = (torch.arange(T)[None] < n.cpu()[:, None]).reshape(-1).numpy()  # the norm of an all-zero row has no slope to compare
    close("dx", g["dx"][torch.from_numpy(live).cuda()], g_ref["dx"][live])
    gs_ref = decay_scan_grad_ref(q, k, v, a, S0, n, do=g["dx"].view(B, T, H, d))
    for i in ("dq", "dk", "dv"):
        close(i, gs[i], gs_ref[i])
    close("dS0", gs["dS0"], gs_ref["dS0"], 2.0 ** -18)
    o1_ref, S1_ref = decay_scan_ref(one["q"], one["k"], one["v"], a, S)
    close("o1", o1, o1_ref)
    close("S1", state, S1_ref, 2.0 ** -18)


def test_autograd_through_the_layer():
    """As a torch.autograd.Function, captured into a graph while an eager graph of the same leaves lives."""
    P = prism()

    class Layer(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, a, w, gate):
            B, T, H, d = q.shape
            o, _ = P.prism_decay_scan_fwd(q, k, v, a, want_state=False)
            y, m, r = P.prism_group_norm_fwd(o.view(B * T, -1), H, w, None, gate, activation="silu")
            ctx.save_for_backward(q, k, v, a, w, gate, o, m, r)
            return y

        @staticmethod
        def backward(ctx, dy):
            q, k, v, a, w, gate, o, m, r = ctx.saved_tensors
            B, T, H, d = q.shape
            g = P.prism_group_norm_bwd(o.view(B * T, -1), H, m, r, w, None, gate, dy=dy.contiguous(), activation="silu")
            gs = P.prism_decay_scan_bwd(q, k, v, a, dO=g["dx"].view(B, T, H, -1), want_dS0=False)
            return gs["dq"], gs["dk"], gs["dv"], None, g["dweight"], g["dgate"]

    x = layer_inputs(3, 1, 200, 4, 2, 64)
    leaves = [x[i].clone().requires_grad_(True) for i in ("q", "k", "v", "weight", "gate")]
    q, k, v, w, gate = leaves

    def loss():
        return (Layer.apply(q, k, v, x["decay"], w, gate).float() * x["dy"].float()).sum()

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        eager = torch.autograd.grad(loss(), leaves)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        captured = torch.autograd.grad(loss(), leaves)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(eager, captured):
        assert torch.equal(a, b)

    # the same layer from differentiable torch operations in 64 bits
    ref = [t.detach().double().requires_grad_(True) for t in leaves]
    Q, K, V, W, Gt = ref
    K, V = K.repeat_interleave(2, 2), V.repeat_interleave(2, 2)
    t = torch.arange(200, device="cuda", dtype=torch.float64)
    gap = t[:, None] - t
    M = torch.where(gap >= 0, x["decay"].double()[:, None, None] ** gap.clamp(min=0), 0.0)
    o = torch.einsum("hij,bihk,bjhk,bjhv->bihv", M, Q, K, V).reshape(200, 4, 64)
    z = (o - o.mean(-1, keepdim=True)) / (o.var(-1, unbiased=False, keepdim=True) + 1e-5).sqrt()
    y = z.reshape(200, 256) * W * torch.nn.functional.silu(Gt)
    want = torch.autograd.grad((y * x["dy"].double()).sum(), ref)
    # o is rounded to bf16 between the stages (2^-8), the norm's derivative and the scan's gradients round
    # once more each, two roundings inside: below 6 x 2^-8
    for a, b in zip(eager, want):
        assert (a.double() - b).norm() <= 6 * 2.0 ** -8 * b.norm()


def test_streaming_with_the_output_norm():
    """The chunk stream's outputs through the gated per-head norm, against the oracles of both; and the same
    layer on the decay scan, whose chunks chain through S_final."""
    import oracle
    from delta_rule_sequence_b200.stream import StreamingScan, head_norm
    from delta_rule_sequence_b200.workloads import WORKLOADS, make_inputs

    P = prism()
    wl = WORKLOADS["gdn"].with_(B=2, H=2, T=3 * 64, s0_std=0.02)
    x = make_inputs(wl, seed=3)
    d = {n: None if t is None else t.cuda() for n, t in x.items()}
    g = torch.Generator().manual_seed(5)
    gate = torch.randn(2, wl.T, 2, 128, generator=g).bfloat16().cuda()
    w = (1 + 0.2 * torch.randn(256, generator=g)).cuda()
    s = StreamingScan(d["S0"], norm_fn=head_norm(w))
    plain = StreamingScan(d["S0"])
    raw, outs = [], []
    for t in range(0, wl.T, 64):
        c = {n: None if v is None or n == "S0" else v[:, t:t + 64].contiguous() for n, v in d.items()}
        args = (c["q"], c["k"], c["v"], c["alpha"], c["beta"])
        outs.append(s.step(*args, gate=gate[:, t:t + 64]))
        raw.append(plain.step(*args))
    torch.cuda.synchronize()
    o_ref, _ = oracle.scan_ref(**x)
    raw = torch.cat(raw, 1)
    err = np.abs(raw.double().cpu().numpy() - o_ref)
    assert (err <= 2e-2 * (1 + np.abs(o_ref))).all()
    y_ref, _, _ = group_norm_ref(raw.reshape(-1, 1, 256), 2, w, None, gate.reshape(-1, 1, 256), activation="silu")
    y = torch.cat(outs, 1).double().cpu().numpy().reshape(y_ref.shape)
    assert np.linalg.norm(y - y_ref) <= 2.0 ** -8 * np.linalg.norm(y_ref)  # rounded once

    a = torch.tensor([0.9, 0.99], device="cuda")
    whole, S_whole = P.prism_decay_scan_fwd(d["q"], d["k"], d["v"], a, d["S0"])
    S, parts = d["S0"], []
    for t in range(0, wl.T, 64):
        o, S = P.prism_decay_scan_fwd(d["q"][:, t:t + 64], d["k"][:, t:t + 64], d["v"][:, t:t + 64], a, S)
        parts.append(o)
    torch.cuda.synchronize()
    o_ref, S_ref = decay_scan_ref(d["q"], d["k"], d["v"], a, d["S0"])
    for got, ref, lim in ((whole, o_ref, 2.0 ** -7), (torch.cat(parts, 1), o_ref, 2.0 ** -7), (S_whole, S_ref, 2.0 ** -18),
                          (S, S_ref, 2.0 ** -18)):
        assert np.linalg.norm(got.double().cpu().numpy() - ref) <= lim * np.linalg.norm(ref)
