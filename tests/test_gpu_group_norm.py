"""The channels-last group norm on the GPU against its fp64 oracle.

Tolerances.  All arithmetic is fp32 from the inputs' exact values.  xh = (x - mean) rstd: the mean has an error of a
few 2^-24 |x|max, the same goes for x - mean, and rstd is off by a few 2^-24 relative; activations and their
slopes are within 2^-20 of max(1, |z|).  So z, y and the gradients' terms are within 2^-18 of
(1 + |x|max rstd) (1 + the term's factors): TERM below, with |x|max rstd for the offset inputs.  bf16 results are
rounded once more, 2^-8 relative.  Sums over n terms (dweight, dbias) add n 2^-24 of the sum of absolute terms at most.
"""
import numpy as np
import pytest
import torch

from oracle.group_norm import group_norm_grad_ref, group_norm_ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def prism():
    from delta_rule_sequence_b200 import prism as P

    return P


def make(seed, N, S, C, io, gate, affine, mean=0.3, std=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return {"x": (mean + std * r(N, S, C)).to(io).cuda(), "dy": r(N, S, C).to(io).cuda(),
            "gate": r(N, S, C).to(io).cuda() if gate else None,
            "weight": (1 + 0.3 * r(C)).cuda() if affine else None, "bias": (0.3 * r(C)).cuda() if affine else None}


def near(name, got, ref, scale, io, term=2.0 ** -18):
    got = got.double().cpu().numpy()
    assert got.shape == ref.shape and np.isfinite(got).all(), name
    tol = term * scale + (2.0 ** -8 * np.abs(ref) if io == BF else 0)
    err = np.abs(got - ref)
    assert (err <= tol).all(), f"{name}: {(err > tol).sum()} of {err.size} off, worst {(err / tol).max():.3g} of the tolerance"


def run_and_check(x, G, activation, eps=1e-5, flat=False):
    P = prism()
    args = (x["weight"], x["bias"], x["gate"])
    io = x["x"].dtype
    y, mean, rstd = P.prism_group_norm_fwd(x["x"], G, *args, eps=eps, activation=activation)
    got = P.prism_group_norm_bwd(x["x"], G, mean, rstd, *args, dy=x["dy"], activation=activation)
    torch.cuda.synchronize()
    ref, m, r = group_norm_ref(x["x"], G, *args, eps=eps, activation=activation)
    N, S, C = x["x"].shape
    big = np.abs(x["x"].double().cpu().numpy()).max()
    cond = (1 + big * r)[:, None, :, None] * np.ones((1, S, 1, C // G))
    cond = cond.reshape(N, S, C)
    w = np.ones(C) if x["weight"] is None else np.abs(x["weight"].double().cpu().numpy())
    gate = np.ones(1) if x["gate"] is None else 1 + np.abs(x["gate"].double().cpu().numpy())
    dy = np.abs(x["dy"].double().cpu().numpy())
    near("mean", mean, m, 1 + big, F32, 2.0 ** -21)
    near("rstd", rstd, r, r * (1 + big * r), F32, 2.0 ** -20)
    near("y", y, ref, cond * (1 + w) * gate, io)
    g = group_norm_grad_ref(x["x"], G, *args, eps=eps, activation=activation, dy=x["dy"])
    assert set(got) == {"dx"} | {"d" + n for n in ("gate", "weight", "bias") if x[n] is not None}
    # dx: (dn - mean(dn) - xh mean(dn xh)) rstd with |xh| up to sqrt(n): every term bounded by cond^2 max|dy|
    xh = cond * (1 + w) * gate
    near("dx", got["dx"], g["dx"], 4 * xh ** 2 * dy.max() * np.repeat(r[:, None, :], C // G, axis=2).reshape(N, 1, C), io)
    if x["gate"] is not None:
        near("dgate", got["dgate"], g["dgate"], xh * (1 + dy), io)
    for n in ("dweight", "dbias"):
        if n in got:
            near(n, got[n], g[n], (dy * gate * xh).sum((0, 1)), F32)
    return y, mean, rstd, got


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("activation", ["none", "silu", "gelu"])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("N,S,C,G", [(37, 1, 256, 4), (3, 50, 96, 8)])
def test_activations_and_gates(io, activation, gate, N, S, C, G):
    run_and_check(make(1, N, S, C, io, gate, True), G, activation)


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("N,S,C,G", [
    (1, 1, 8, 1), (1, 1, 1, 1), (5, 1, 3, 3), (7, 1, 7, 1), (700, 1, 64, 2), (2000, 1, 32, 4), (4, 1, 640, 5),  # 128 wide
    (9, 1, 300, 3), (3, 1, 258, 2), (2, 1, 2048, 1), (2, 1, 4096, 1), (2, 1, 1032, 1), (5, 1, 129, 1), (2, 1, 5000, 2),
    (1, 2, 8, 1), (2, 15, 24, 24), (2, 16, 17, 1), (1, 33, 40, 4), (3, 100, 320, 32), (1, 1000, 30, 5), (2, 40, 2080, 13),
    (1, 20, 4104, 3), (2, 7, 2056, 257), (1, 5000, 8, 2), (130, 3, 6, 2), (1, 17, 700, 7),
])
def test_shapes(io, N, S, C, G):
    run_and_check(make(2, N, S, C, io, True, True), G, "silu")


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("S", [1, 64])
def test_no_weights(io, S):
    run_and_check(make(3, 6, S, 64, io, False, False), 4, "gelu")


@pytest.mark.parametrize("S", [1, 64])
@pytest.mark.parametrize("only", ["weight", "bias"])
def test_weight_or_bias_alone(S, only):
    x = make(11, 5, S, 96, BF, True, True)
    x["bias" if only == "weight" else "weight"] = None
    run_and_check(x, 6, "silu")


@pytest.mark.parametrize("S", [1, 300])
def test_mean_far_above_the_deviation(S):
    run_and_check(make(4, 4, S, 64, F32, False, True, mean=1000.0, std=0.5), 2, "none")


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("S", [1, 40])
def test_constant_groups(io, S):
    """No deviation at all: rstd = 1 / sqrt(eps), xh = 0."""
    x = make(5, 3, S, 32, io, False, True)
    x["x"].fill_(2.5)
    y, mean, rstd = prism().prism_group_norm_fwd(x["x"], 4, x["weight"], x["bias"], eps=1e-3)
    torch.cuda.synchronize()
    assert (mean == 2.5).all()
    np.testing.assert_allclose(rstd.cpu().numpy(), 1e-3 ** -0.5, rtol=2e-6)
    assert torch.equal(y.float(), x["bias"].to(io).float().expand_as(y.float()))


@pytest.mark.parametrize("S", [1, 40])
def test_large_gates_and_values_stay_finite(S):
    x = make(6, 3, S, 64, F32, True, True)
    x["gate"].mul_(1e4)
    P = prism()
    for act in ("silu", "gelu"):
        y, mean, rstd = P.prism_group_norm_fwd(x["x"], 4, x["weight"], x["bias"], x["gate"], activation=act)
        got = P.prism_group_norm_bwd(x["x"], 4, mean, rstd, x["weight"], x["bias"], x["gate"], dy=x["dy"], activation=act)
        assert torch.isfinite(y).all() and all(torch.isfinite(t).all() for t in got.values())


def test_a_sample_with_nan_leaves_the_others():
    for S in (1, 30):
        x = make(7, 5, S, 64, BF, True, True)
        want = prism().prism_group_norm_fwd(x["x"], 2, x["weight"], x["bias"], x["gate"], activation="silu")
        x["x"][2, 0, 3] = float("nan")  # group 0 of sample 2
        got = prism().prism_group_norm_fwd(x["x"], 2, x["weight"], x["bias"], x["gate"], activation="silu")
        torch.cuda.synchronize()
        keep = [0, 1, 3, 4]
        assert torch.equal(got[0][keep], want[0][keep]) and torch.equal(got[0][2, :, 32:], want[0][2, :, 32:])
        assert torch.isnan(got[0][2, :, :32]).all()


def test_dimensions_between_samples_and_channels_are_positions():
    x = make(8, 3, 24, 32, BF, False, True)
    a = prism().prism_group_norm_fwd(x["x"], 4, x["weight"], x["bias"])
    b = prism().prism_group_norm_fwd(x["x"].view(3, 4, 6, 32), 4, x["weight"], x["bias"])
    c = prism().prism_group_norm_fwd(x["x"].view(72, 32), 4, x["weight"], x["bias"])
    d = prism().prism_group_norm_fwd(x["x"].view(72, 1, 32), 4, x["weight"], x["bias"])
    torch.cuda.synchronize()
    assert torch.equal(a[0].view(-1), b[0].view(-1)) and torch.equal(c[0].view(-1), d[0].view(-1))
    assert c[1].shape == (72, 4)


def test_empty():
    P = prism()
    w = torch.ones(8, device="cuda")
    for shape in ((0, 8), (0, 3, 8), (2, 0, 8)):
        x = torch.zeros(shape, dtype=BF, device="cuda")
        y, mean, rstd = P.prism_group_norm_fwd(x, 2, w, w)
        got = P.prism_group_norm_bwd(x, 2, mean, rstd, w, w, dy=x)
        torch.cuda.synchronize()
        assert y.shape == x.shape and (got["dweight"] == 0).all() and (got["dbias"] == 0).all()


def test_same_bits_every_time_captured_and_on_streams():
    P = prism()
    for S, N in ((1, 3000), (200, 4)):
        x = make(9, N, S, 96, BF, True, True)

        def calls(stream=None):
            y, m, r = P.prism_group_norm_fwd(x["x"], 6, x["weight"], x["bias"], x["gate"], activation="silu", stream=stream)
            return [y, m, r, *P.prism_group_norm_bwd(x["x"], 6, m, r, x["weight"], x["bias"], x["gate"], dy=x["dy"],
                                                     activation="silu", stream=stream).values()]

        want = calls()
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(3)]
        outs = [calls(streams[i % 3]) for i in range(6)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for o in outs for a, b in zip(o, want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = calls()
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_wrappers_refuse():
    P = prism()
    x = make(10, 4, 3, 32, BF, True, True)
    with pytest.raises(ValueError):
        P.prism_group_norm_fwd(x["x"], 5)
    with pytest.raises(ValueError):
        P.prism_group_norm_fwd(x["x"], 4, activation="tanh")
    with pytest.raises(ValueError):
        P.prism_group_norm_fwd(x["x"].transpose(0, 1), 4)
    with pytest.raises(TypeError):
        P.prism_group_norm_fwd(x["x"], 4, x["weight"].to(BF))
    with pytest.raises(TypeError):
        P.prism_group_norm_fwd(x["x"].half(), 4)
    with pytest.raises(P.PrismError):
        P.prism_group_norm_fwd(x["x"], 4, y=x["x"])
    with pytest.raises(P.PrismError):
        P.prism_group_norm_fwd(x["x"], 4, eps=-1.0)


def test_a_larger_workspace_and_given_outputs():
    P = prism()
    for S in (1, 70):
        x = make(12, 4, S, 64, BF, False, True)
        want, m, r = P.prism_group_norm_fwd(x["x"], 4, x["weight"], x["bias"])
        ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")  # any contents
        y = torch.full_like(x["x"], float("nan"))
        got, m2, r2 = P.prism_group_norm_fwd(x["x"], 4, x["weight"], x["bias"], y=y, workspace=ws)
        g = P.prism_group_norm_bwd(x["x"], 4, m, r, x["weight"], x["bias"], dy=x["dy"])
        ws.fill_(255)
        g2 = P.prism_group_norm_bwd(x["x"], 4, m, r, x["weight"], x["bias"], dy=x["dy"], workspace=ws)
        torch.cuda.synchronize()
        assert got is y and torch.equal(y, want) and torch.equal(m, m2) and torch.equal(r, r2)
        assert all(torch.equal(g[n], g2[n]) for n in g)


def test_rows_behind_31_bits():
    """Every row on its own: the last rows of 2.3e9 elements have the bits that they have alone."""
    P = prism()
    N, C, G = (1 << 20) + 5, 17 * 128, 17
    g = torch.Generator(device="cuda").manual_seed(13)
    x, dy = (torch.randn(N, C, generator=g, device="cuda", dtype=BF) for _ in range(2))
    y, mean, rstd = P.prism_group_norm_fwd(x, G, gate=dy, activation="silu")
    got = P.prism_group_norm_bwd(x, G, mean, rstd, gate=x, dy=dy, activation="silu")
    y1, m1, r1 = P.prism_group_norm_fwd(x[-999:], G, gate=dy[-999:], activation="silu")
    got1 = P.prism_group_norm_bwd(x[-999:], G, m1, r1, gate=x[-999:], dy=dy[-999:], activation="silu")
    assert torch.equal(y[-999:], y1) and torch.equal(mean[-999:], m1) and torch.equal(rstd[-999:], r1)
    assert all(torch.equal(got[n][-999:], got1[n]) for n in got1)


def test_positions_behind_31_bits():
    """The last of three samples of 2^20 x 768 against 64 bits."""
    P = prism()
    N, S, C, G = 3, 1 << 20, 768, 8
    g = torch.Generator(device="cuda").manual_seed(14)
    x, dy = (torch.randn(N, S, C, generator=g, device="cuda", dtype=BF) for _ in range(2))
    y, mean, rstd = P.prism_group_norm_fwd(x, G)
    dx = P.prism_group_norm_bwd(x, G, mean, rstd, dy=dy)["dx"]
    xd = x[2].double().view(S, G, C // G)
    m = xd.mean((0, 2))
    r = (xd.var((0, 2), unbiased=False) + 1e-5).rsqrt()
    big = xd.abs().max()
    assert ((mean[2] - m).abs() <= 2.0 ** -21 * (1 + big)).all()
    assert ((rstd[2] - r).abs() <= 2.0 ** -20 * r * (1 + big * r)).all()
    xh = (xd - m[:, None]) * r[:, None]
    del xd
    cond = float(1 + big * r.max())
    tol = 2.0 ** -18 * cond * 2
    assert ((y[2].view(S, G, -1) - xh).abs() <= tol + 2.0 ** -8 * xh.abs()).all()
    d = dy[2].double().view(S, G, C // G)
    ref = (d - d.mean((0, 2))[:, None] - xh * (d * xh).mean((0, 2))[:, None]) * r[:, None]
    tol = 2.0 ** -18 * 4 * (2 * cond) ** 2 * float(d.abs().max() * r.max())
    assert ((dx[2].view(S, G, -1) - ref).abs() <= tol + 2.0 ** -8 * ref.abs()).all()
