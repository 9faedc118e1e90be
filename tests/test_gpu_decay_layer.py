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
