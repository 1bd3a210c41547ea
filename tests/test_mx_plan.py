"""The packed product's division among pairs of thread blocks
(lutq_mx_gemm_plan), checked on the host for devices and partitions of all
sizes: no more pairs than the multiprocessors hold, every tile taken, and
where pairs share tiles by K (each then takes one tile and ends) as many
groups of pairs as tiles."""
import pytest

import dequant_gemv_group_b200 as lq

SHAPES = [(m, n, k) for m in (1, 17, 64, 128, 129, 192, 193, 256, 300, 513, 4099)
          for n in (1, 256, 512, 1024, 2304, 4096, 9472, 19333, 28672, 76200)
          for k in (32, 1024, 4096, 8192, 14336, 28672)]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("sms", [2, 4, 8, 16, 18, 24, 32, 36, 48, 64, 70, 96, 132, 148, 160])
def test_every_tile_is_taken(fmt, sms):
    for m, n, k in SHAPES:
        p = lq.lutq_mx_gemm_plan(m, n, k, fmt, sms)
        assert p["rows"] in (256, 512) and p["split"] in (1, 2, 4)
        assert 1 <= p["pairs"] <= sms // 2 and p["pairs"] % p["split"] == 0
        assert p["tokens"] % 32 == 0 and min(m, 256) <= p["tokens"] <= 256
        tiles = -(-n // p["rows"]) * -(-m // 256)
        if p["split"] > 1:
            assert p["pairs"] == tiles * p["split"], (m, n, k, p)
            assert -(-k // 256) >= p["split"]
        if p["rows"] == 512:
            assert p["tokens"] <= 192 and p["split"] == 1


def test_plan_on_a_whole_device():
    """The divisions that the measured shapes have."""
    assert lq.lutq_mx_gemm_plan(4096, 14336, 4096, "mxfp4", 148) == dict(
        rows=256, tokens=256, split=1, pairs=74)
    assert lq.lutq_mx_gemm_plan(133, 28672, 8192, "nvfp4", 148) == dict(
        rows=512, tokens=160, split=1, pairs=56)
    assert lq.lutq_mx_gemm_plan(128, 512, 14336, "mxfp4", 148) == dict(
        rows=256, tokens=128, split=4, pairs=8)
    assert lq.lutq_mx_gemm_plan(512, 4096, 14336, "mxfp4", 148) == dict(
        rows=256, tokens=256, split=2, pairs=64)


def test_refusals():
    for a in ((0, 8, 32), (-1, 8, 32), (1, 0, 32), (1, 8, 48), (1 << 30, 8, 32)):
        with pytest.raises(lq.LutqError):
            lq.lutq_mx_gemm_plan(*a, "mxfp4", 148)
    with pytest.raises(lq.LutqError):
        lq.lutq_mx_gemm_plan(1, 8, 32, "mxfp4", 0)
    with pytest.raises(ValueError):
        lq.lutq_mx_gemm_plan(1, 8, 32, "fp4", 148)
    assert lq.lib.lutq_mx_gemm_plan(1, 8, 32, 0, 148, None) == 1
