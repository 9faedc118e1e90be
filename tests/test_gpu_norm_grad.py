"""The group norm's gradients on the GPU, term by term (tests/norm_checks.py)."""
import pytest
import torch

from tests.norm_checks import check_grads
from tests.test_norm_checks import make

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def prism():
    from delta_rule_sequence_b200 import prism as P

    return P


def run_and_check(x, G, activation, gated=True, affine=True, eps=1e-5):
    P = prism()
    x = {n: t.cuda() for n, t in x.items()}
    args = (x["weight"] if affine else None, x["bias"] if affine else None, x["gate"] if gated else None)
    _, mean, rstd = P.prism_group_norm_fwd(x["x"], G, *args, eps=eps, activation=activation)
    got = P.prism_group_norm_bwd(x["x"], G, mean, rstd, *args, dy=x["dy"], activation=activation)
    check_grads(got, x["x"], G, mean, rstd, *args, dy=x["dy"], activation=activation)


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("activation", ["none", "silu", "gelu"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("N,S,C,G", [(37, 1, 256, 4), (3, 50, 96, 8), (2, 30, 30, 5), (6, 1, 45, 3)])
def test_activations_and_gates(io, activation, gated, N, S, C, G):
    run_and_check(make(3, N, S, C, io, 0.3, 1.0), G, activation, gated)


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("mean,std", [(0.3, 1.0), (1000.0, 4.0)])
@pytest.mark.parametrize("N,S,C,G", [
    (1, 1, 8, 1), (700, 1, 64, 2), (2000, 1, 32, 4), (4, 1, 640, 5), (3, 1, 258, 2), (2, 1, 2048, 1), (2, 1, 4096, 1),
    (5, 1, 129, 1), (2, 1, 5000, 2), (2, 15, 24, 24), (2, 16, 17, 1), (3, 100, 320, 32), (1, 1000, 30, 5), (2, 40, 2080, 13),
    (1, 20, 4104, 3), (2, 7, 2056, 257), (1, 5000, 8, 2), (130, 3, 6, 2), (400, 70, 16, 2), (1, 17, 700, 7),
])
def test_shapes(io, mean, std, N, S, C, G):
    run_and_check(make(4, N, S, C, io, mean, std), G, "silu")


@pytest.mark.parametrize("S", [1, 300])
def test_mean_far_above_the_deviation(S):
    run_and_check(make(5, 4, S, 64, F32, 1000.0, 0.5), 2, "none", gated=False)


@pytest.mark.parametrize("S", [1, 64])
def test_no_weights(S):
    run_and_check(make(6, 6, S, 64, BF, 0.3, 1.0), 4, "gelu", gated=False, affine=False)


def test_positions_behind_31_bits():
    """The last of three samples of 2^20 x 768 (2.4e9 elements)."""
    P = prism()
    N, S, C, G = 3, 1 << 20, 768, 8
    g = torch.Generator(device="cuda").manual_seed(14)
    x, dy = (torch.randn(N, S, C, generator=g, device="cuda", dtype=BF) for _ in range(2))
    _, mean, rstd = P.prism_group_norm_fwd(x, G)
    dx = P.prism_group_norm_bwd(x, G, mean, rstd, dy=dy)["dx"][2]
    # one group at a time: its reference's intermediates are 0.8 GB each
    for k in (0, 7):
        cut = slice(k * 96, (k + 1) * 96)
        check_grads({"dx": dx[None, :, cut]}, x[2:, :, cut].contiguous(), 1, mean[2:, k:k + 1], rstd[2:, k:k + 1],
                    dy=dy[2:, :, cut].contiguous())
