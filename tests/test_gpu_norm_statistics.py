"""Means and deviations of the group norm over many positions with a mean far above the deviation.

A sample that is one tile (300 samples leave each one) has up to S / RL positions in a thread, RL = 256 / (vectors of
a position) row lanes.  Tolerances, u = 2^-24: a thread's mean is rounded once (u |mean|), the merges of a group's
threads and of its tiles round theirs once more each; a block of 16 positions adds 16 deviations with an error of at most
16 u 16 max|x - mean|, 16 u max|x - mean| for each of them.  So the mean is within 4 u max|x| + 64 u max|x - mean|.
The sum of squares: a block of b positions behind n others has the squares q about their mean, and adds q - w t, where
w t <= q b / (n + b) (w is a sum of b terms, w^2 <= b q), so at least q n / (n + b); its b + 3 operations on q and w t are
off by 2 (b + 3) u q, and the result by 2 (b + 3) (1 + b / n) u relative.  The blocks are (n, b) = (1, 4), (5, 16),
(21, 16), ...: 70, 160, 67 and fewer, each of its own share of the sum, so 160 u at most.  Its additions to the sum,
S / (16 RL), and the merges', 256 / 32 + 16 each, come to it: K in all, and rstd is within (K / 2 + 4) u relative.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def prism():
    from delta_rule_sequence_b200 import prism as P

    return P


def inputs(seed, N, S, C, io, mean, std):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(N, S, C, generator=g, device="cuda").mul_(std).add_(mean).to(io)


def check(x, G, eps=1e-5):
    N, S, C = x.shape
    y, mean, rstd = prism().prism_group_norm_fwd(x, G, eps=eps)
    vector = 16 // x.element_size() if C % (16 // x.element_size()) == 0 else 1
    lanes = max(1, 256 // (C // vector))
    K = 160 + S / (16 * lanes) + 2 * (256 / 32 + 16)
    for n in sorted({0, N // 2, N - 1}):
        d = x[n].double().view(S, G, C // G)
        big = d.abs().amax((0, 2))
        m = d.mean((0, 2))
        d = d - m[:, None]
        dev = d.abs().amax((0, 2))
        r = (d.square().mean((0, 2)) + eps).rsqrt()
        mean_tol = U * (4 * big + 64 * dev)
        assert ((mean[n] - m).abs() <= mean_tol).all(), ((mean[n] - m).abs() / mean_tol).max()
        rstd_tol = (K / 2 + 4) * U
        assert ((rstd[n] - r).abs() <= rstd_tol * r).all(), ((rstd[n] / r - 1).abs() / rstd_tol).max()
        z = d * r[:, None]
        tol = (r * mean_tol)[:, None] + (rstd_tol + 4 * U + (2.0 ** -8 if x.dtype == BF else 0)) * z.abs() + 1e-30
        assert ((y[n].view(S, G, -1) - z).abs() <= tol).all()
    return y, mean, rstd


@pytest.mark.parametrize("io,N,S,C,G,mean,std", [
    (F32, 300, 16384, 256, 256, 1000.0, 0.5),  # one channel a group, four row lanes of 4096 positions
    (F32, 300, 4096, 1024, 8, 1e4, 1.0),       # one row lane
    (F32, 300, 30000, 3, 3, 100.0, 1.0),       # single channels
    (BF, 300, 2048, 2048, 2048, 100.0, 4.0),
    (F32, 1, 1 << 20, 4, 4, 1000.0, 0.5),      # one sample, many tiles
    (F32, 300, 2000, 8, 2, 0.0, 1.0),
])
def test_mean_far_above_the_deviation_over_many_positions(io, N, S, C, G, mean, std):
    check(inputs(1, N, S, C, io, mean, std), G)


@pytest.mark.parametrize("C", [64, 3])
def test_a_first_value_far_from_the_others(C):
    x = inputs(2, 300, 4000, C, F32, 0.0, 1.0)
    x[:, 0] = 1e4
    check(x, C)


@pytest.mark.parametrize("C", [64, 3])
@pytest.mark.parametrize("value", [1000.0 / 3, 0.1, -7e6])
def test_equal_values_have_exactly_their_mean(C, value):
    x = torch.full((300, 3000, C), value, device="cuda")
    y, mean, rstd = prism().prism_group_norm_fwd(x, C, eps=1e-3)
    assert (mean == x[0, 0, 0]).all() and (y == 0).all()
    assert ((rstd - 1e-3 ** -0.5).abs() <= 4 * U * 1e-3 ** -0.5).all()
