"""Hidden values next to a rounding border, in each of the experts' kernels.

All sums here are exact (few bits), and the down matrix is the identity, so y
is the quantized hidden value itself.  What is left is silu(g) * u in fp32:
exp off by at most 2 units of 2^-23, and four roundings of 2^-24 each, 2^-21 in
all, so a hidden value that lies 2^-21 of itself or more from the border
between two bf16 values is on the right side of it.  The inputs are values 2^-21 to 2^-19
from borders that decide a 4-bit level, gates from -8 to -88.
"""
import numpy as np
import pytest
import torch

from oracle import mx_oracle as O
from test_gpu_experts import lq  # noqa: F401

pytestmark = pytest.mark.gpu

D = F = 128
USED = [i for i in range(32) if i % 16]  # (positions 0, 16, ... hold the 6 that sets x's scales)


def _silu64(g):
    return g / (1.0 + np.exp(-g))


def _candidates():
    """(g, u) with g in steps of 1/256, u an odd number up to 335 times a power of two."""
    g = -np.arange(8 * 256, 84 * 256) / 256.0
    odd = np.arange(1, 336, 2).astype(np.float64)
    h = np.abs(_silu64(g))[:, None] * odd[None]
    m = np.frexp(h)[0] * 2  # in [1, 2)
    out = []
    # where the nearest of 2^k (1, 1.5, 2) changes: 1.25, to the even level 1, and 1.75, to 2; and,
    # between .5 and 1, .75 to 1: the bf16 value in the middle and its neighbour round apart
    for border, top in ((1.25 + 2.0 ** -8, 1.0), (1.75 - 2.0 ** -8, 1.0), (1.5 - 2.0 ** -8, 0.5)):
        off = np.abs(m / border - 1.0)
        for i, j in zip(*np.nonzero((off >= 2.0 ** -21) & (off <= 2.0 ** -19))):
            e = np.frexp(h[i, j])[1] - 1
            out.append((g[i], odd[j], np.log2(top) - e))
    out.sort()  # gates far below zero first
    out.insert(0, (-88.0, 1.0, 119.0))  # 1 + exp(88) is beyond 2^126
    return out


def _levels(total, places):
    """Codes of E2M1 levels at `places` that add up to total (a multiple of 0.5)."""
    codes = np.zeros(64, np.uint8)
    sign, left, at = (8 if total < 0 else 0), abs(total), iter(places)
    for i in range(7, 0, -1):
        while left >= O.LEVELS[i]:
            codes[next(at)] = sign | i
            left -= O.LEVELS[i]
    assert left == 0
    return codes


def _matrices():
    """Gate and up codes [F, D] with the scale of each 32 positions as an exponent, and (g, u)."""
    cand = _candidates()
    gate, up = np.zeros((F, D), np.uint8), np.zeros((F, D), np.uint8)
    ge, ue = np.zeros((F, 2), int), np.zeros((F, 2), int)
    g, u = np.zeros(F), np.zeros(F)
    for f in range(F):
        if f % 16 == 0:
            g[f], odd, e = 32.0, 3.0, -4.0           # h = 6 sets the block's scale
        elif cand:
            g[f], odd, e = cand.pop(0)
        else:
            continue
        u[f] = odd * 2.0 ** e
        # x is 4 there: g = 4 (2^-3 S1 + 2^-9 S2)
        fine = np.sign(g[f]) * (abs(g[f]) * 256 % 64) / 2
        s1 = (g[f] - fine * 2.0 ** -7) * 2
        gate[f, :64] = _levels(s1, USED) | _levels(fine, [32 + i for i in USED])
        ge[f] = -3, -9
        up[f, :64] = _levels(odd / 2, USED)
        ue[f] = e - 1, e - 1
    return gate, up, ge, ue, g, u


def _pack(lq, codes, exponents, fmt):  # noqa: F811
    pair = torch.from_numpy(codes[:, 0::2] | (codes[:, 1::2] << 4)).cuda()
    per = 32 // O.BLOCK[fmt]
    if fmt == "mxfp4":
        s = np.full((F, D // 32), 127, np.uint8)
        s[:, :2] = exponents + 127
        return lq.lutq_mx_pack(pair, torch.from_numpy(s).cuda(), fmt)
    rows = torch.exp2(torch.from_numpy(exponents[:, 0]).float())
    s = np.zeros((F, D // 16), np.uint8)
    s[:, :2 * per] = np.repeat(np.where(exponents - exponents[:, :1] == 0, 0x38, 0x08), per, 1)
    return lq.lutq_mx_pack(pair, torch.from_numpy(s).cuda(), fmt, rows.cuda())


# one token; more pairs an expert than the kernel of few tokens takes; block pairs
@pytest.mark.parametrize("t", [1, 20, 40])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_hidden_values_beside_a_border(lq, fmt, t):  # noqa: F811
    gate, up, ge, ue, g, u = _matrices()
    one = torch.zeros(F, D)
    one[torch.arange(F), torch.arange(D)] = 6.0      # level 6, scale 1
    down = lq.lutq_mx_quantize(one.bfloat16().cuda(), fmt)
    x = torch.zeros(t, D)
    x[:, :64] = 4.0
    x[:, :64:16] = 6.0
    w = torch.full((t, 1), 1 / 6)
    ids = torch.zeros(t, 1, dtype=torch.int32)
    y = lq.lutq_mx_experts(x.cuda(), ids.cuda(), w.cuda(), _pack(lq, gate, ge, fmt).unsqueeze(0),
                           _pack(lq, up, ue, fmt).unsqueeze(0), down.unsqueeze(0), F, fmt)
    want = O.values(*O.quantize(O.to_bf16(_silu64(g) * u)[None], fmt), fmt)[0]
    assert len(set(want[16:32])) > 1
    # (times 6 exactly, and the weight 1 / 6: back within some units of 2^-24)
    y = (y.double().cpu().numpy() * 4).round() / 4
    wrong = np.nonzero((y != want).any(0))[0]
    assert not len(wrong), [(int(f), g[f], u[f], y[0, f], want[f]) for f in wrong[:8]]
