"""The decay scan at the edges of what its documentation allows: most batches and heads, overlapping and reordered views,
one tensor in several roles, padded batches without a token.  Tolerances as in tests/decay_checks.py."""
import pytest
import torch

from tests.decay_checks import check_bwd, check_fwd, make

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def prism():
    from delta_rule_sequence_b200 import prism as P

    return P


def run(x, dO, dS=None):
    P = prism()
    o, S = P.prism_decay_scan_fwd(x["q"], x["k"], x["v"], x["decay"], x["S0"], x["lengths"])
    got = P.prism_decay_scan_bwd(x["q"], x["k"], x["v"], x["decay"], x["S0"], x["lengths"], dO=dO, dS_final=dS)
    torch.cuda.synchronize()
    return o, S, got


def check(x, dO, dS=None):
    o, S, got = run(x, dO, dS)
    check_fwd(x, o, S)
    check_bwd(x, dO, dS, got)


def part(x, b, h):
    """Batches b and heads h (slices) of the inputs."""
    return {"q": x["q"][b, :, h], "k": x["k"][b, :, h], "v": x["v"][b, :, h], "decay": x["decay"][h],
            "S0": None if x["S0"] is None else x["S0"][b, h], "lengths": None if x["lengths"] is None else x["lengths"][b]}


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("B,H", [(65535, 1), (1, 65535)])
def test_most_batches_and_heads(io, B, H):
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    T, d = 3, 32
    x = {"q": r(B, T, H, d).to(io), "k": (r(B, T, H, d) * d ** -0.5).to(io), "v": r(B, T, H, d).to(io),
         "decay": torch.rand(H, generator=g, device="cuda"), "S0": r(B, H, d, d),
         "lengths": torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)}
    if B == 1:
        x["lengths"].fill_(T)
    dO = r(B, T, H, d).to(io)
    o, S, got = run(x, dO)
    P = prism()
    state = x["S0"].clone()
    o1 = P.prism_decay_step(x["q"][:, :1], x["k"][:, :1], x["v"][:, :1], x["decay"], state)
    for i in (0, 777, 65528):
        b, h = (slice(i, i + 7), slice(None)) if B > 1 else (slice(None), slice(i, i + 7))
        y = part(x, b, h)
        check_fwd(y, o[b, :, h], S[b, h])
        check_bwd(y, dO[b, :, h], None, {n: t[b, h] if n == "dS0" else t[b, :, h] for n, t in got.items()})
        one = dict(y, lengths=None, **{n: y[n][:, :1] for n in "qkv"})
        check_fwd(one, o1[b, :, h], state[b, h])


@pytest.mark.parametrize("io", [BF, F32])
def test_head_major_views(io):
    """[B, heads, T, d] in memory, as many models keep them."""
    x = make(2, 2, 200, 4, 2, 64, 32, io, ragged=True)
    dO = torch.randn(2, 200, 4, 32, generator=torch.Generator().manual_seed(3)).to(io).cuda()
    y = dict(x, **{n: x[n].transpose(1, 2).contiguous().transpose(1, 2) for n in "qkv"})
    a, b = run(x, dO), run(y, dO)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and all(torch.equal(a[2][n], b[2][n]) for n in a[2])
    check(y, dO)


@pytest.mark.parametrize("io", [BF, F32])
def test_overlapping_windows(io):
    """Token t's key is values 16 t to 16 t + 63 of a signal: strides are smaller than the width."""
    x = make(4, 1, 300, 2, 2, 64, 64, io, S0=False)
    signal = torch.randn(2 * (16 * 299 + 64), generator=torch.Generator().manual_seed(5)).mul(0.125).to(io).cuda()
    x["k"] = signal.as_strided((1, 300, 2, 64), (1 << 20, 16, 16 * 299 + 64, 1))
    dO = torch.randn(1, 300, 2, 64, generator=torch.Generator().manual_seed(6)).to(io).cuda()
    check(x, dO)


@pytest.mark.parametrize("io", [BF, F32])
def test_one_tensor_in_several_roles(io):
    x = make(7, 2, 150, 2, 2, 64, 64, io)
    x["q"] = x["v"] = x["k"]
    check(x, x["k"], x["S0"])


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("T", [1, 3000])
def test_a_padded_batch_without_a_token(io, T):
    x = make(8, 3, T, 2, 1, 64, 128, io)
    x["lengths"] = torch.zeros(3, dtype=torch.int32, device="cuda")
    for n in "qkv":
        x[n].fill_(float("nan"))
    dO, dS = torch.full((3, T, 2, 128), float("nan"), dtype=io, device="cuda"), torch.randn(3, 2, 128, 64, device="cuda")
    o, S, got = run(x, dO, dS)
    assert torch.equal(S, x["S0"]) and torch.equal(got["dS0"], dS)
    assert all((t == 0).all() for t in (o, got["dq"], got["dk"], got["dv"]))


@pytest.mark.parametrize("io", [BF, F32])
def test_given_back_into_the_same_state_with_lengths(io):
    """S_final is S0, in segments and with sequences that end in different ones."""
    x = make(9, 4, 2500, 2, 2, 64, 64, io, ragged=True)
    want_o, want_S = prism().prism_decay_scan_fwd(x["q"], x["k"], x["v"], x["decay"], x["S0"], x["lengths"])
    S = x["S0"].clone()
    o, got = prism().prism_decay_scan_fwd(x["q"], x["k"], x["v"], x["decay"], S, x["lengths"], S_final=S)
    torch.cuda.synchronize()
    assert got is S and torch.equal(S, want_S) and torch.equal(o, want_o)


def test_two_graphs_with_one_workspace():
    """Replayed one after the other on one stream, each gives its own results."""
    P = prism()
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    xs = [make(10 + i, 2, 700, 4, 2, 64, 64, ragged=True) for i in range(2)]
    dOs = [torch.randn(2, 700, 4, 64, device="cuda").bfloat16() for _ in range(2)]

    def call(i):
        x = xs[i]
        o, S = P.prism_decay_scan_fwd(x["q"], x["k"], x["v"], x["decay"], x["S0"], x["lengths"], workspace=ws)
        g = P.prism_decay_scan_bwd(x["q"], x["k"], x["v"], x["decay"], x["S0"], x["lengths"], dO=dOs[i], workspace=ws)
        return [o, S, *g.values()]

    want = [call(i) for i in range(2)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(call(i))
    for i in (0, 1, 1, 0, 1):
        graphs[i].replay()
    torch.cuda.synchronize()
    for got, ref in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
