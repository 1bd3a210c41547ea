"""Dequantize: zero rows, and one rounding whatever a checkpoint's row scales are."""
import numpy as np
import pytest
import torch

from oracle import mx_oracle as O
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


@pytest.mark.parametrize("n,k", [(1031, 1056), (3, 64)])
def test_rounded_once(lq, n, k):  # noqa: F811
    """level * E4M3 scale has 6 bits at most, times an fp32 row scale 30: exact in fp64, rounded
    once to each type.  (fp64 -> fp32 -> bf16 differs in about one of 2^17 values.)"""
    g = torch.Generator().manual_seed(n)
    codes = torch.randint(0, 256, (n, k // 2), generator=g).to(torch.uint8)
    scales = torch.randint(0, 0x7f, (n, k // 16), generator=g).to(torch.uint8)
    rows = torch.rand(n, generator=g) + 2.0 ** -3
    rows[0], rows[1] = 0.25, -rows[1]
    # rows made so that 1.5 * rows lies just beside the middle of two values of the type
    mid = torch.arange(1, 65).double()
    for i, bits in ((2, 8), (66, 11)):
        m = torch.floor(mid * 2.0 ** (bits - 1) / 64) * 2.0 ** -bits + 1 + 2.0 ** -bits
        rows[i:i + 64] = torch.nextafter((m / 1.5).float(), torch.tensor(2.0))[:max(0, n - i)]
    c = np.stack([codes.numpy() & 15, codes.numpy() >> 4], -1).reshape(n, k)
    want = O.values(c, scales.numpy(), rows.numpy(), "nvfp4")
    packed = lq.lutq_mx_pack(codes.cuda(), scales.cuda(), "nvfp4", rows.cuda())

    def got(dtype):
        return lq.lutq_mx_dequantize(packed, n, k, "nvfp4", dtype=dtype).double().cpu().numpy()

    np.testing.assert_array_equal(got(torch.float32), want.astype(np.float32).astype(np.float64))
    np.testing.assert_array_equal(got(torch.bfloat16), O.to_bf16(want))
    np.testing.assert_array_equal(got(torch.float16), want.astype(np.float16).astype(np.float64))
    if n > 1000:  # (the inputs tell one rounding from two)
        twice = O.to_bf16(want.astype(np.float32).astype(np.float64))
        assert (twice != O.to_bf16(want)).any()
        assert (want.astype(np.float32).astype(np.float16) != want.astype(np.float16)).any()
