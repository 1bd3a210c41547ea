"""Routing to experts on the GPU against the oracle: ids equal, weights within
their one rounding to fp32 (2^-24 relative) and some units of fp64."""
import numpy as np
import pytest
import torch

from oracle import mx_oracle as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dequant_gemv_group_b200 as m
    return m


def _check(lq, z, k, bias=None, status=0, **kw):
    st = lq.new_status()
    ids, w = lq.lutq_route(z.cuda(), k, bias=None if bias is None else bias.cuda(), status=st, **kw)
    ri, rw = O.route(z.double().numpy(), k, bias=None if bias is None else bias.double().numpy(),
                     **kw)
    assert ids.dtype == torch.int32 and w.dtype == torch.float32
    np.testing.assert_array_equal(ids.cpu().numpy(), ri)
    np.testing.assert_allclose(w.double().cpu().numpy(), rw, rtol=2.0 ** -24 * 1.001, atol=1e-45)
    assert int(st.item()) == status


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("t,e,k", [(1, 1, 1), (1, 8, 2), (3, 32, 32), (5, 33, 4), (37, 64, 8),
                                   (4, 127, 6), (9, 256, 8), (2, 500, 10), (3, 1024, 16)])
def test_plain(lq, dtype, score, t, e, k):
    z = (torch.randn(t, e, generator=torch.Generator().manual_seed(e + k)) * 2).to(dtype)
    _check(lq, z, k, score=score, renormalize=(e + k) % 2 == 0, scale=1.0 if k < 8 else 2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,groups,kept,best,k", [(16, 4, 1, 1, 4), (160, 8, 3, 1, 6),
                                                  (256, 8, 4, 2, 8), (60, 3, 2, 2, 5),
                                                  (32, 32, 7, 2, 7), (1024, 2, 1, 2, 32),
                                                  (24, 24, 24, 1, 3), (21, 7, 7, 2, 21)])
def test_groups_and_bias(lq, score, e, groups, kept, best, k):
    g = torch.Generator().manual_seed(e + groups)
    z = torch.randn(29, e, generator=g) * 1.5
    bias = torch.randn(e, generator=g) * 0.2
    for b in (None, bias):
        _check(lq, z, k, bias=b, score=score, groups=groups, top_groups=kept, group_best=best,
               renormalize=True, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties(lq, score):
    """Equal logits: the lowest expert first, whatever lane it is in; groups the same way."""
    z = torch.zeros(4, 96)
    z[1, 40:] = 1.0
    z[2, ::3] = -1.0
    z[3] = (torch.arange(96) // 7 % 3).float()
    _check(lq, z, 8, score=score)
    _check(lq, z, 8, score=score, groups=8, top_groups=3, group_best=2)
    _check(lq, z.to(torch.bfloat16), 32, score=score, renormalize=True)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_masked_rows(lq, score, dtype):
    """-infinity masks an expert; a row may have fewer than top_k left, or none; the type's lowest
    value is an ordinary (tiny) score."""
    g = torch.Generator().manual_seed(3)
    z = torch.randn(8, 64, generator=g)
    z[0] = -np.inf
    z[1, 1:] = -np.inf
    z[2, :60] = -np.inf
    z[3, ::2] = -np.inf
    z[4] = torch.finfo(dtype).min
    z[5, 5:] = torch.finfo(dtype).min
    z[6, :32] = -np.inf
    z = z.to(dtype)
    bias = torch.randn(64, generator=g)
    for b in (None, bias):
        for kw in (dict(), dict(groups=4, top_groups=2), dict(groups=8, top_groups=2, group_best=2)):
            for renorm in (False, True):
                _check(lq, z, 6, bias=b, score=score, renormalize=renorm, **kw)


def test_extreme_logits(lq):
    z = torch.tensor([[1e4, -1e4, 0.0, 80.0], [-800.0, -700.0, 700.0, 800.0],
                      [1e-30, 0.0, -1e-30, 2e-30]])
    _check(lq, z, 3, score="softmax")
    _check(lq, z, 3, score="sigmoid")


def test_near_ties_need_64_bits(lq):
    """Scores 1 + n 2^-23 apart in the logits: fp32 scores would tie, fp64 ones do not."""
    z = 1.0 + torch.arange(64).flip(0).float().repeat(2, 1) * 2.0 ** -23
    z[1] = z[1].flip(0)
    _check(lq, z, 8, score="sigmoid")
    _check(lq, z, 8, score="softmax")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("gap", [2.0 ** -23, 3e-7, 1e-6, 4e-6, 1.7e-5, 1e-4])
def test_close_calls(lq, score, gap):
    """Logits, biases and group sums about as far apart as 32-bit scores can tell, and closer."""
    g = torch.Generator().manual_seed(int(1 / gap))
    z = torch.randn(40, 16, generator=g).repeat_interleave(64, 1)
    z = z + gap * torch.randint(-3, 4, (40, 1024), generator=g)
    _check(lq, z, 20, bias=(gap * torch.randint(-2, 3, (1024,), generator=g)).float(), score=score)
    base = torch.randn(200, 8, generator=g).repeat_interleave(8, 1)
    z = base + gap * torch.randint(-3, 4, (200, 64), generator=g)
    bias = (gap * torch.randint(-2, 3, (64,), generator=g)).float()
    for b in (None, bias):
        for kw in (dict(), dict(groups=8, top_groups=3, group_best=2), dict(groups=4, top_groups=1)):
            _check(lq, z, 8, bias=b, score=score, renormalize=True, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_nonfinite_reported(lq, score):
    z = torch.randn(3, 40, generator=torch.Generator().manual_seed(1))
    z[1, 7] = np.nan
    _check(lq, z, 4, score=score, status=5)
    z[1, 7], z[2, 9] = 0.0, np.inf
    _check(lq, z, 4, score=score, status=5)


def test_many_tokens_empty_and_unaligned(lq):
    z = torch.randn(5001, 128, generator=torch.Generator().manual_seed(2))
    _check(lq, z, 4)
    ids, w = lq.lutq_route(torch.empty(0, 128, device="cuda"), 4)
    assert ids.shape == w.shape == (0, 4)
    buf = torch.randn(3 * 50 + 1, device="cuda")
    part = buf[1:].view(3, 50)            # 4-byte aligned only
    a, b = lq.lutq_route(part, 5), lq.lutq_route(part.clone(), 5)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
