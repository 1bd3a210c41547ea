"""An expert with more (token, choice) pairs than there are tokens: a token may
name an expert more than once."""
import pytest
import torch

from test_gpu_experts import Layer, _close, _inputs, lq  # noqa: F401

pytestmark = pytest.mark.gpu

# packed tokens in narrow tiles; in tiles of 128; block pairs; the kernel of few tokens
CASES = [(1, 4, 64), (2, 4, 64), (16, 4, 4), (16, 1, 2), (20, 2, 3), (32, 3, 4), (33, 8, 4),
         (50, 16, 4), (64, 20, 5), (70, 30, 6), (40, 4, 4), (150, 5, 3), (4, 64, 32), (8, 64, 40),
         (2, 40, 9)]


def _ids(t, e, k, how):
    if how == "one":                                    # all pairs to one expert
        return torch.full((t, k), e - 1, dtype=torch.int32)
    ids = torch.randint(-1, e, (t, k), generator=torch.Generator().manual_seed(t + k)).int()
    ids[:, : (3 * k + 3) // 4] = e // 2                 # most of them, the others anywhere
    return ids


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("how", ["one", "most"])
@pytest.mark.parametrize("t,e,k", CASES)
def test_repeated_ids(lq, fmt, how, t, e, k):  # noqa: F811
    d, f = 288, 160
    layer = Layer(lq, e, d, f, fmt, seed=t)
    x, _ = _inputs(t, e, k, d, seed=e)
    x *= torch.exp2(torch.arange(t) % 7 - 3.0).unsqueeze(1).cuda().bfloat16()  # scales differ by row
    ids = _ids(t, e, k, how).cuda()
    w = torch.rand(t, k, generator=torch.Generator().manual_seed(k)).cuda()
    nb = lq.lutq_mx_experts_workspace_bytes(t, k, e, d, f, fmt)
    space = torch.full((nb + 4096,), 255, dtype=torch.uint8, device="cuda")
    y = layer.run(x, ids, w, workspace=space[:nb])
    _close(y, *layer.reference(x, ids, w))
    assert (space[nb:] == 255).all()
