"""The decay scan on the GPU against its fp64 oracle: forward, backward, single tokens."""
import numpy as np
import pytest
import torch

from oracle.decay_scan import decay_scan_grad_ref, decay_scan_ref
from tests.decay_checks import check, check_bwd, check_fwd, make

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def prism():
    from delta_rule_sequence_b200 import prism as P

    return P


def fwd(x, **kw):
    out = prism().prism_decay_scan_fwd(x["q"], x["k"], x["v"], x["decay"], x["S0"], x["lengths"], **kw)
    torch.cuda.synchronize()
    return out


def bwd(x, dO, dS=None, **kw):
    out = prism().prism_decay_scan_bwd(x["q"], x["k"], x["v"], x["decay"], x["S0"], x["lengths"], dO=dO, dS_final=dS, **kw)
    torch.cuda.synchronize()
    return out


def grads_of(seed, x):
    B, T, H, _ = x["q"].shape
    g = torch.Generator().manual_seed(seed)
    dv, dk = x["v"].shape[-1], x["q"].shape[-1]
    return (torch.randn(B, T, H, dv, generator=g).to(x["q"].dtype).cuda(), 0.3 * torch.randn(B, H, dv, dk, generator=g).cuda())


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("dk,dv", [(32, 32), (64, 64), (128, 128), (32, 128), (128, 32), (64, 128), (128, 64), (32, 64)])
def test_forward_widths(io, dk, dv):
    x = make(1, 2, 300, 4, 2, dk, dv, io)
    check_fwd(x, *fwd(x))


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("T", [1, 2, 31, 63, 64, 65, 127, 128, 129, 255, 256, 257, 700])
def test_forward_lengths(io, T):
    x = make(2, 1, T, 3, 1, 64, 64, io, S0=T % 2 == 0)
    check_fwd(x, *fwd(x))


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("T", [1, 2, 64, 65, 127, 128, 129, 257, 600])
def test_backward_lengths(io, T):
    x = make(3, 1, T, 4, 2, 64, 32, io, S0=T % 2 == 0)
    dO, dS = grads_of(4, x)
    check_bwd(x, dO, dS, bwd(x, dO, dS))


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("dk,dv", [(32, 32), (64, 64), (128, 128), (32, 128), (128, 32), (64, 128), (128, 64)])
@pytest.mark.parametrize("Hkv", [4, 1])
def test_backward_widths(io, dk, dv, Hkv):
    x = make(5, 2, 290, 4, Hkv, dk, dv, io)
    dO, dS = grads_of(6, x)
    check_bwd(x, dO, dS, bwd(x, dO, dS))


def test_backward_without_state_gradients():
    x = make(7, 2, 150, 2, 2, 64, 64, S0=False)
    dO, _ = grads_of(8, x)
    got = bwd(x, dO, want_dS0=False)
    assert got["dS0"] is None
    check_bwd(x, dO, None, got)


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_padded_batch_ignores_what_is_behind_the_end(io, d):
    x = make(9, 6, 400, 2, 1, d, d, io, ragged=True)
    n = x["lengths"]
    n[1], n[2], n[3] = 0, 1, 128
    dO, dS = grads_of(10, x)
    for b in range(6):  # NaN and infinities in the padding reach nothing
        for t, bad in ((x["q"], float("nan")), (x["k"], float("inf")), (x["v"], float("nan")), (dO, float("-inf"))):
            t[b, n[b]:] = bad
    o, S = fwd(x)
    check_fwd(x, o, S)
    got = bwd(x, dO, dS)
    check_bwd(x, dO, dS, got)
    for b in range(6):
        for t in (o, got["dq"], got["dk"], got["dv"]):
            assert (t[b, n[b]:] == 0).all()
    assert torch.equal(S[1], x["S0"][1])  # no tokens: the entry state, bit for bit
    assert torch.equal(got["dS0"][1], dS[1])


def test_lengths_out_of_range_are_clamped():
    x = make(11, 3, 130, 2, 2, 64, 64)
    x["lengths"] = torch.tensor([-5, 1000, 130], dtype=torch.int32, device="cuda")
    o, S = fwd(x)
    x["lengths"] = torch.tensor([0, 130, 130], dtype=torch.int32, device="cuda")
    o2, S2 = fwd(x)
    assert torch.equal(o, o2) and torch.equal(S, S2)


@pytest.mark.parametrize("decay", [[0.0, 0.0], [1.0, 1.0], [1e-30, 0.5], [1 - 2.0 ** -24, 2.0 ** -100]])
@pytest.mark.parametrize("io", [BF, F32])
def test_extreme_decays(decay, io):
    x = make(12, 1, 333, 2, 2, 64, 64, io, decay=decay)
    check_fwd(x, *fwd(x))
    dO, dS = grads_of(13, x)
    check_bwd(x, dO, dS, bwd(x, dO, dS))


@pytest.mark.parametrize("io", [BF, F32])
def test_strided_views(io):
    """q, k, v as views of one projection [B, T, (H + 2 Hkv), d], and with batch and token exchanged."""
    x = make(14, 2, 200, 4, 2, 64, 64, io)
    fused = torch.cat([x["q"], x["k"], x["v"]], dim=2).contiguous()
    y = dict(x, q=fused[:, :, :4], k=fused[:, :, 4:6], v=fused[:, :, 6:])
    z = dict(x, **{n: x[n].transpose(0, 1).contiguous().transpose(0, 1) for n in "qkv"})
    dO, dS = grads_of(15, x)
    want, wantg = fwd(x), bwd(x, dO, dS)
    for w in (y, z):
        got, gotg = fwd(w), bwd(w, dO, dS)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        for n in wantg:
            assert torch.equal(gotg[n], wantg[n]), n


@pytest.mark.parametrize("io", [BF, F32])
def test_many_segments_and_few_sequences(io):
    x = make(16, 1, 5000, 1, 1, 64, 64, io, decay=[0.9995])
    check_fwd(x, *fwd(x))
    dO, dS = grads_of(17, x)
    check_bwd(x, dO, dS, bwd(x, dO, dS))


@pytest.mark.parametrize("io,dk,dv", [(BF, 64, 64), (BF, 128, 64), (BF, 64, 128), (BF, 128, 128), (BF, 32, 64), (F32, 64, 64)])
@pytest.mark.parametrize("ragged", [False, True])
def test_long_walks(io, dk, dv, ragged):
    """Enough sequences that one CTA walks many chunks; sampled sequences against the oracle."""
    x = make(40, 40, 1500, 4, 2, dk, dv, io, ragged=ragged)
    dO, dS = grads_of(41, x)
    o, S = fwd(x)
    got = bwd(x, dO, dS)
    assert all(torch.isfinite(t).all() for t in (o, S, *got.values()))
    for b in (0, 7, 39):
        one = {n: t if t is None or n == "decay" else t[b:b + 1] for n, t in x.items()}
        check_fwd(one, o[b:b + 1], S[b:b + 1])
        check_bwd(one, dO[b:b + 1], dS[b:b + 1], {n: t[b:b + 1] for n, t in got.items()})


def test_many_sequences():
    x = make(18, 40, 70, 8, 8, 32, 32)
    check_fwd(x, *fwd(x))
    dO, dS = grads_of(19, x)
    check_bwd(x, dO, dS, bwd(x, dO, dS))


def test_resumes_from_its_own_state_in_place():
    x = make(20, 2, 513, 3, 3, 128, 64)
    whole, S = fwd(x)
    first = dict(x, **{n: x[n][:, :200].contiguous() for n in "qkv"})
    rest = dict(x, **{n: x[n][:, 200:] for n in "qkv"})
    state = x["S0"].clone()
    o1, _ = fwd(dict(first, S0=state), S_final=state)
    o2, _ = fwd(dict(rest, S0=state), S_final=state)  # S_final is S0
    check_fwd(x, torch.cat([o1, o2], 1), state)


def test_outputs_given_by_the_caller_and_no_state():
    x = make(21, 1, 100, 2, 2, 64, 64)
    o = torch.full((1, 100, 2, 64), float("nan"), dtype=BF, device="cuda")
    got, S = fwd(x, o=o, want_state=False)
    assert got is o and S is None
    check_fwd(x, o, None)


def test_no_tokens():
    x = make(22, 2, 0, 2, 2, 64, 64)
    o, S = fwd(x)
    assert o.numel() == 0 and torch.equal(S, x["S0"])
    _, S = fwd(dict(x, S0=None))
    assert (S == 0).all()
    dO, dS = grads_of(23, x)
    assert torch.equal(bwd(x, dO, dS)["dS0"], dS)
    assert (bwd(x, dO)["dS0"] == 0).all()


def test_agrees_with_the_delta_rule_scan_without_erase():
    P = prism()
    x = make(24, 2, 300, 2, 2, 64, 64, decay=[0.9, 0.99])
    alpha = x["decay"].expand(2, 300, 2).contiguous()
    u, w = x["v"].unsqueeze(3).contiguous(), x["k"].unsqueeze(3).contiguous()
    o, S = P.prism_scan_fwd(x["q"], x["k"], None, alpha, torch.zeros_like(alpha), u, w, x["S0"])
    o2, S2 = fwd(x)
    ref, refS = decay_scan_ref(**x)
    mass, massS = decay_scan_ref(**{n: t if n in ("decay", "lengths") or t is None else t.float().abs() for n, t in x.items()})
    # each within its own tolerance of the exact value, so within their sum of each other: the delta-rule
    # scan's 2e-2 (1 + |r|), and this scan's 2^-8 (|r| + M) for o, 2^-14 M for the state (decay_checks)
    for a, b, r, own in ((o, o2, ref, 2.0 ** -8 * (np.abs(ref) + mass)), (S, S2, refS, 2.0 ** -14 * massS)):
        err = np.abs(a.double().cpu().numpy() - b.double().cpu().numpy())
        worst = (err / (2e-2 * (1 + np.abs(r)) + own)).max()
        assert worst <= 1, worst


def test_same_bits_every_time_and_on_other_streams():
    x = make(25, 2, 900, 4, 2, 128, 128, ragged=True)
    dO, dS = grads_of(26, x)
    want, wantg = fwd(x), bwd(x, dO, dS)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    outs = []
    for i in range(9):  # calls in flight at the same time on several streams
        s = streams[i % 3]
        outs.append(prism().prism_decay_scan_fwd(x["q"], x["k"], x["v"], x["decay"], x["S0"], x["lengths"], stream=s))
        outs.append(prism().prism_decay_scan_bwd(x["q"], x["k"], x["v"], x["decay"], x["S0"], x["lengths"], dO=dO,
                                                 dS_final=dS, stream=s))
    torch.cuda.synchronize()
    for o in outs:
        if isinstance(o, dict):
            assert all(torch.equal(o[n], wantg[n]) for n in wantg)
        else:
            assert torch.equal(o[0], want[0]) and torch.equal(o[1], want[1])


def test_captured_and_replayed():
    P = prism()
    x = make(27, 2, 300, 4, 4, 64, 64)
    dO, dS = grads_of(28, x)
    S = x["S0"].clone()
    one = {n: x[n][:, :1] for n in "qkv"}

    def calls():
        a = P.prism_decay_scan_fwd(x["q"], x["k"], x["v"], x["decay"], x["S0"])
        b = P.prism_decay_scan_bwd(x["q"], x["k"], x["v"], x["decay"], x["S0"], dO=dO, dS_final=dS)
        c = P.prism_decay_step(one["q"], one["k"], one["v"], x["decay"], S)
        return [*a, *b.values(), c, S]

    calls()
    torch.cuda.synchronize()
    S.copy_(x["S0"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = calls()
    y = make(29, 2, 300, 4, 4, 64, 64)  # other inputs in the captured buffers
    for n in "qkv":
        x[n].copy_(y[n])
    S.copy_(x["S0"])
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in outs]
    S.copy_(x["S0"])
    want = calls()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("dk,dv", [(32, 32), (64, 64), (128, 128), (32, 128), (128, 32), (64, 128)])
@pytest.mark.parametrize("B,H,Hkv", [(1, 1, 1), (3, 4, 2), (70, 8, 1)])
def test_step(io, dk, dv, B, H, Hkv):
    x = make(30, B, 1, H, Hkv, dk, dv, io)
    S = x["S0"].clone()
    o = prism().prism_decay_step(x["q"], x["k"], x["v"], x["decay"], S)
    torch.cuda.synchronize()
    # all in fp32: the output is rounded once, each sum has dk + 2 operations
    ref, refS = decay_scan_ref(**x)
    mass, massS = decay_scan_ref(**{n: t if n in ("decay", "lengths") or t is None else t.float().abs() for n, t in x.items()})
    check("S", S, refS, massS, False)
    err = np.abs(o.double().cpu().numpy() - ref)
    assert (err <= (2.0 ** -8 * np.abs(ref) if io == BF else 0) + 2.0 ** -16 * mass).all()


def test_steps_follow_the_scan():
    x = make(31, 2, 20, 4, 2, 64, 128)
    S = x["S0"].clone()
    outs = [prism().prism_decay_step(x["q"][:, t:t + 1], x["k"][:, t:t + 1], x["v"][:, t:t + 1], x["decay"], S) for t in range(20)]
    torch.cuda.synchronize()
    check_fwd(x, torch.cat(outs, 1), S)


def test_wrappers_refuse():
    P = prism()
    x = make(32, 2, 10, 4, 2, 64, 64)
    q, k, v, a = (x[n] for n in ("q", "k", "v", "decay"))
    with pytest.raises(TypeError):
        P.prism_decay_scan_fwd(q.half(), k.half(), v.half(), a)
    with pytest.raises(TypeError):
        P.prism_decay_scan_fwd(q, k.float(), v, a)
    with pytest.raises(TypeError):
        P.prism_decay_scan_fwd(q, k, v, a.double())
    with pytest.raises(ValueError):
        P.prism_decay_scan_fwd(q, k[:, :, :1], v, a)
    with pytest.raises(ValueError):
        P.prism_decay_scan_fwd(q[:, :, :3], k, v, a[:3])  # 2 heads do not divide 3
    with pytest.raises(ValueError):
        P.prism_decay_scan_fwd(q.transpose(2, 3).contiguous().transpose(2, 3), k, v, a)  # width not dense
    with pytest.raises(ValueError):
        P.prism_decay_scan_fwd(q, k[:, :1].expand(2, 10, 2, 64), v, a)  # stride 0 over tokens
    with pytest.raises(TypeError):
        P.prism_decay_scan_fwd(q, k, v, a, lengths=torch.ones(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(P.PrismError):
        P.prism_decay_scan_fwd(q[..., :48].contiguous(), k[..., :48].contiguous(), v, a)  # width 48
    with pytest.raises(P.PrismError):
        P.prism_decay_scan_fwd(q, k, v, a, o=q.view(2, 10, 4, 64))  # o is q
    with pytest.raises(P.PrismError):
        P.prism_decay_step(q, k, v, a, x["S0"])  # 10 tokens
    with pytest.raises(ValueError):
        P.prism_decay_scan_bwd(q, k, v, a, dO=torch.empty(2, 4, 10, 64, dtype=BF, device="cuda").transpose(1, 2))


def test_a_stalled_pipeline_gives_up():
    """The loads are not issued: every wait of the tensor-core kernels runs out, the kernels return and the
    status says so; the next call works."""
    P = prism()
    lib = P.load_library()
    x = make(33, 1, 400, 2, 2, 128, 64)
    dO, dS = grads_of(34, x)
    want = fwd(x)
    old = lib.prism_debug_set_flags(256)
    try:
        P.prism_decay_scan_fwd(x["q"], x["k"], x["v"], x["decay"], x["S0"])
        assert P.prism_query_device_status(None) == P.PRISM_ERR_TIMEOUT
        P.prism_decay_scan_bwd(x["q"], x["k"], x["v"], x["decay"], x["S0"], dO=dO, dS_final=dS)
        assert P.prism_query_device_status(None) == P.PRISM_ERR_TIMEOUT
    finally:
        lib.prism_debug_set_flags(old)
    assert P.prism_query_device_status(None) == P.PRISM_OK
    got = fwd(x)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("io", [BF, F32])
def test_a_workspace_with_any_contents(io):
    x = make(35, 2, 700, 4, 2, 64, 64, io, ragged=True)
    dO, dS = grads_of(36, x)
    want, wantg = fwd(x), bwd(x, dO, dS)
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")  # every float a NaN
    got = fwd(x, workspace=ws)
    ws.fill_(255)
    gotg = bwd(x, dO, dS, workspace=ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert all(torch.equal(gotg[n], wantg[n]) for n in wantg)
    with pytest.raises(prism().PrismError):
        fwd(x, workspace=ws[:256])


def test_first_calls_of_a_process_under_capture():
    """No warm-up before the capture: what a call looks up on first use is allowed there."""
    import os
    import subprocess
    import sys

    code = """
import torch
from delta_rule_sequence_b200 import prism as P
q, k, v = (torch.randn(1, 200, 2, 64, device="cuda").bfloat16() for _ in range(3))
a = torch.full((2,), 0.9, device="cuda")
S = torch.zeros(1, 2, 64, 64, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    o, _ = P.prism_decay_scan_fwd(q, k, v, a)
    gr = P.prism_decay_scan_bwd(q, k, v, a, dO=o)
    P.prism_decay_step(q[:, :1], k[:, :1], v[:, :1], a, S)
    y, m, r = P.prism_group_norm_fwd(o.view(200, 128), 2, activation="silu")
    n = P.prism_group_norm_bwd(o.view(1, 200, 128), 2, m[:1], r[:1], dy=o.view(1, 200, 128))
g.replay()
torch.cuda.synchronize()
want, _ = P.prism_decay_scan_fwd(q, k, v, a)
torch.cuda.synchronize()
assert torch.equal(o, want) and torch.isfinite(gr["dq"].float()).all()
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=240)
    assert r.returncode == 0, r.stderr[-2000:]


def test_offsets_beyond_31_bits():
    """2^20 tokens of 17 x 128: the operands' last elements lie behind 2^31 (and the fp32 partial gradients of the
    shared head behind 2^33 bytes).  With a decay of 1/2 a token's reach ends after 512 (2^-512 times its mass), so
    the last 1024 tokens alone give the last 512 tokens' results."""
    T, H, d = 1 << 20, 17, 128
    g = torch.Generator(device="cuda").manual_seed(37)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=BF)  # noqa: E731
    x = {"q": r(1, T, H, d), "k": r(1, T, 1, d) * d ** -0.5, "v": r(1, T, 1, d), "decay": torch.full((H,), 0.5, device="cuda"),
         "S0": None, "lengths": None}
    dO = r(1, T, H, d)
    o, S = fwd(x)
    got = bwd(x, dO)
    tail = {n: t[:, -1024:].contiguous() if n in "qkv" else t for n, t in x.items()}
    mass = {n: t.float().abs() if n in "qkv" else t for n, t in tail.items()}
    ref, m = decay_scan_ref(**tail), decay_scan_ref(**mass)
    check("o", o[:, -512:], ref[0][:, -512:], m[0][:, -512:], True)
    check("S_final", S, ref[1], m[1], False)
    args = {"do": dO[:, -1024:], "dS_final": None}
    ref = decay_scan_grad_ref(**tail, **args)
    m = decay_scan_grad_ref(**mass, do=args["do"].float().abs(), dS_final=None)
    for n in ("dq", "dk", "dv"):
        check(n, got[n][:, -512:], ref[n][:, -512:], m[n][:, -512:], True)
