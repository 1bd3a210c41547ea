"""Group scores whose two best biased scores cancel: their sum is far smaller
than what it is the sum of, and 32-bit sums of them do not tell the order."""
import numpy as np
import pytest
import torch

from test_gpu_route import _check, lq  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [1.0, 16.0, 4096.0, 1e6])
@pytest.mark.parametrize("e,groups,kept", [(64, 32, 11), (64, 16, 5), (256, 8, 3), (40, 4, 2)])
def test_biases_that_cancel(lq, score, size, e, groups, kept):  # noqa: F811
    g = torch.Generator().manual_seed(e + groups + int(size))
    z = torch.randn(300, e, generator=g) * 0.3
    # a group's two best: one with +size, one with -size; the others far below
    bias = torch.full((groups, e // groups), -4 * size)
    bias[:, 0], bias[:, 1] = size, -size
    _check(lq, z, 4, bias=bias.flatten(), score=score, groups=groups, top_groups=kept,
           group_best=2, renormalize=True)


def test_large_biases_that_do_not_cancel(lq):  # noqa: F811
    """Experts left out by a bias of -1e9, and one group far above the others."""
    g = torch.Generator().manual_seed(5)
    z = torch.randn(200, 64, generator=g)
    bias = torch.randn(64, generator=g) * 0.1
    bias[::5] = -1e9
    bias[16:24] += 1e4
    for best in (1, 2):
        _check(lq, z, 6, bias=bias, score="sigmoid", groups=8, top_groups=3, group_best=best)
    assert np.isfinite(bias.numpy()).all()
