"""Dequantize: zero rows."""
import pytest
import torch

from test_gpu_mx import lq  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_zero_rows(lq, fmt):  # noqa: F811
    """What quantize makes of no rows, dequantize takes back."""
    for shape in ((0, 64), (0, 7, 64), (3, 0, 64)):
        w = torch.empty(*shape, dtype=torch.bfloat16, device="cuda")
        back = lq.lutq_mx_dequantize(lq.lutq_mx_quantize(w, fmt), shape[-2], 64, fmt)
        assert back.shape == shape and back.dtype == torch.bfloat16
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    for n, k in ((0, 48), (0, 0), (-1, 64), (8, 64)):
        with pytest.raises(lq.LutqError):
            lq.lutq_mx_dequantize(none, n, k, fmt)
