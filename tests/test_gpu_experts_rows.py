"""The experts' layer sums the pairs' rows in fp32 at every batch size.

The bound is that of test_gpu_experts.py for a single token: the sums' errors,
hidden values next to a bf16 border, and the one rounding of y.  It has no
term for a rounding of the rows, so where a token's rows cancel, rows rounded
to 16 bits are beyond it.
"""
import pytest
import torch

from test_gpu_experts import Layer, _close, _inputs, lq  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("t,e,k", [(64, 2, 2), (65, 2, 2), (65, 4, 4), (300, 5, 4), (1100, 3, 3)])
def test_rows_are_not_rounded(lq, fmt, t, e, k):  # noqa: F811
    d, f = 320, 32
    layer = Layer(lq, e, d, f, fmt, seed=t + e)
    x, z = _inputs(t, e, k, d, seed=k)
    ids = z.argsort(1)[:, :k].int().contiguous() if k <= e else None
    w = torch.randn(t, k, generator=torch.Generator().manual_seed(t)).cuda()
    _close(layer.run(x, ids, w), *layer.reference(x, ids, w, batch=1))


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_precision_does_not_depend_on_the_type(lq, fmt):  # noqa: F811
    """The same tokens as bf16 and as fp32: y differs by bf16's rounding of y alone."""
    t, e, k, d, f = 200, 3, 3, 256, 64
    layer = Layer(lq, e, d, f, fmt, seed=1)
    x, z = _inputs(t, e, k, d, seed=2)
    ids = z.argsort(1)[:, :k].int().contiguous()
    w = torch.randn(t, k, generator=torch.Generator().manual_seed(3)).cuda()
    assert torch.equal(layer.run(x, ids, w), layer.run(x.float(), ids, w).bfloat16())
