"""The group norm over samples without positions."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(2, 0, 8), (3, 4, 0, 8)])
def test_statistics_over_nothing_are_nan(shape):
    """Not what the memory held before."""
    from delta_rule_sequence_b200 import prism as P

    x = torch.zeros(shape, device="cuda")
    for _ in range(3):
        old = [torch.full((shape[0], 2), 7.0, device="cuda") for _ in range(8)]
        del old
        y, mean, rstd = P.prism_group_norm_fwd(x, 2)
        torch.cuda.synchronize()
        assert y.shape == shape and mean.shape == rstd.shape == (shape[0], 2)
        assert torch.isnan(mean).all() and torch.isnan(rstd).all()
    y, mean, rstd = P.prism_group_norm_fwd(torch.zeros(0, 5, 8, device="cuda"), 2)
    assert mean.shape == (0, 2)
