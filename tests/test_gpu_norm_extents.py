"""The group norm at the edges of what its documentation allows: most channels, groups, samples and positions, one tensor in
several roles, and other activations' extremes.  Forward bounds as in tests/test_gpu_norm_statistics.py, gradients as in
tests/norm_checks.py."""
import pytest
import torch

from tests.norm_checks import activation_of, check_grads
from tests.test_gpu_norm_statistics import check

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def prism():
    from delta_rule_sequence_b200 import prism as P

    return P


def normal(seed, *shape, io=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(io)


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("N,S,C,G", [
    (2, 5, 1 << 20, 1 << 20),    # one channel a group: 2048 groups of a block's columns
    (2, 5, 1 << 20, 1),
    (3, 2, (1 << 20) - 1, 3),
    (1, (1 << 22) + 3, 4, 2),
    (5000, 3, 24, 3),
])
def test_most_channels_groups_and_positions(io, N, S, C, G):
    x, dy = normal(1, N, S, C, io=io), normal(2, N, S, C, io=io)
    y, mean, rstd = check(x, G)
    got = prism().prism_group_norm_bwd(x, G, mean, rstd, dy=dy)
    for n in sorted({0, N - 1}):
        check_grads({"dx": got["dx"][n:n + 1]}, x[n:n + 1], G, mean[n:n + 1], rstd[n:n + 1], dy=dy[n:n + 1])


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("N,C,G", [(1 << 24, 8, 1), (3, 1 << 20, 1 << 20), (3, 1 << 20, 1 << 13)])
def test_most_rows_and_groups_of_a_row(io, N, C, G):
    """Samples of the same rows alone, and the first and last of them against 64 bits."""
    x, dy = normal(3, N, C, io=io), normal(4, N, C, io=io)
    w, b = normal(5, C, io=F32), normal(6, C, io=F32)
    y, mean, rstd = prism().prism_group_norm_fwd(x, G, w, b, dy, activation="silu")
    got = prism().prism_group_norm_bwd(x, G, mean, rstd, w, b, dy, dy=dy, activation="silu")
    for cut in (slice(0, 3), slice(N - 3, N)):
        c = x[cut]
        y1, m1, r1 = prism().prism_group_norm_fwd(c, G, w, b, dy[cut], activation="silu")
        g1 = prism().prism_group_norm_bwd(c, G, m1, r1, w, b, dy[cut], dy=dy[cut], activation="silu")
        assert torch.equal(y[cut], y1) and torch.equal(mean[cut], m1) and torch.equal(rstd[cut], r1)
        assert torch.equal(got["dx"][cut], g1["dx"]) and torch.equal(got["dgate"][cut], g1["dgate"])
        check_grads({n: t[:, None] if t.dim() == 2 else t for n, t in g1.items()}, c[:, None], G, m1, r1, w, b,
                    dy[cut][:, None], dy=dy[cut][:, None], activation="silu")
    if N > 1000:  # sums over all rows, in 64 bits
        d = x.double()
        xh = (d - mean.double()) * rstd.double()
        dz = dy.double() * activation_of("silu", dy.double())[0]
        # K additions: a lane's rows, the lanes' parts; K u of the absolute sums, and 2^-20 (1 + |gate|) of each term
        K = N / (148 * 2 * 64) + 300
        for name, t in (("dbias", dz), ("dweight", dz * xh)):
            tol = (K * 2.0 ** -24 * t.abs() + 2.0 ** -20 * (1 + dy.double().abs()) * dy.double().abs() * (1 + xh.abs())).sum(0)
            assert ((got[name] - t.sum(0)).abs() <= tol).all(), name


@pytest.mark.parametrize("S", [1, 60])
def test_one_tensor_in_several_roles(S):
    x = normal(7, 4, S, 96)
    y, mean, rstd = prism().prism_group_norm_fwd(x, 6, gate=x, activation="gelu")
    got = prism().prism_group_norm_bwd(x, 6, mean, rstd, gate=x, dy=x, activation="gelu")
    check_grads(got, x, 6, mean, rstd, gate=x, dy=x, activation="gelu")


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("S", [1, 60])
@pytest.mark.parametrize("activation", ["silu", "gelu"])
def test_far_tails_of_the_activations(io, S, activation):
    """Results and gates from -300 to 300, zeros of either sign among them."""
    t = torch.linspace(-300, 300, 64, device="cuda")
    gate = t.expand(4, S, 64).contiguous().to(io)
    gate[0, 0, :2] = torch.tensor([0.0, -0.0])
    x, dy = normal(8, 4, S, 64, io=io), normal(9, 4, S, 64, io=io)
    for g, bias in ((gate, None), (None, t)):
        args = (None if bias is None else torch.ones(64, device="cuda"), bias, g)
        y, mean, rstd = prism().prism_group_norm_fwd(x, 4, *args, activation=activation)
        got = prism().prism_group_norm_bwd(x, 4, mean, rstd, *args, dy=dy, activation=activation)
        check_grads(got, x, 4, mean, rstd, *args, dy=dy, activation=activation)
        xh = ((x.double().view(4, S, 4, 16) - mean.double().view(4, 1, 4, 1)) * rstd.double().view(4, 1, 4, 1)).view(4, S, 64)
        z = xh if bias is None else xh + bias.double()
        v = z * activation_of(activation, g.double())[0] if g is not None else activation_of(activation, z)[0]
        scale = (1 + z.abs()) * (1 if g is None else 1 + g.double().abs())
        assert ((y - v).abs() <= 2.0 ** -20 * scale + (2.0 ** -8 if io == BF else 0) * v.abs()).all()
