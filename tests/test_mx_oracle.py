"""The oracle of the 4-bit floating-point format against its definition by
other means: exact rational arithmetic, brute force, bytes worked out by hand."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import mx_oracle as O


def test_e4m3_table():
    v = O.e4m3_values()
    assert v[0] == 0 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and v[126] == 448
    assert (np.diff(v) > 0).all() and v[0x38] == 1.0


@pytest.mark.parametrize("x,code", [
    (0.0, 0), (0.25, 0), (0.2500001, 1), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6),
    (5.0, 6), (5.0001, 7), (6.0, 7), (7.9, 7), (-0.0, 8), (-0.75, 10), (-7.0, 15)])
def test_rounding_to_levels(x, code):
    """With 4.0 in the block the mxfp4 scale is 1 (for |x| < 8): the element alone is rounded."""
    v = np.zeros((1, 32))
    v[0, :2] = x, 4.0
    codes, scales, _ = O.quantize(v, "mxfp4")
    assert scales[0, 0] == 127 and codes[0, 0] == code and codes[0, 1] == 6


def test_nvfp4_hand_block():
    # row maximum 8: g = 2^(3 - 10) = 1/128; block maximum 8: s = 8 * 128 / 6 = 170.67 -> 176
    v = np.zeros((1, 32))
    v[0, :4] = 8.0, 1.0, -3.0, 0.3
    v[0, 16] = 2.0 ** -14
    codes, scales, rows = O.quantize(v, "nvfp4")
    assert rows[0] == 1 / 128 and O.e4m3_values()[scales[0, 0]] == 176
    assert list(codes[0, :4]) == [7, 1, 12, 0]     # 5.82 -> 6; .727 -> .5; 2.18 -> 2; .218 -> 0
    # second block: 2^-14 * 128 / 6 = 0.0013, nearer to 2^-9 than to 0; 2^-14 / (2^-9 / 128) = 4
    assert scales[0, 1] == 1 and codes[0, 16] == 6


def _exact_scale(block, row, fmt):
    m = max(abs(Fraction(float(v))) for v in block)
    if fmt == "mxfp4":
        if m == 0:
            return Fraction(1, 2 ** 127)
        e = 0
        while Fraction(2) ** (e + 1) <= m:
            e += 1
        while Fraction(2) ** e > m:
            e -= 1
        return Fraction(2) ** max(e - 2, -127)
    r = max(abs(Fraction(float(v))) for v in row)
    if r == 0:
        return Fraction(0)
    e = 0
    while Fraction(2) ** (e + 1) <= r:
        e += 1
    while Fraction(2) ** e > r:
        e -= 1
    g = Fraction(2) ** max(e - 10, -126)
    t = m / 6 / g
    best = None
    for b, v in enumerate(O.e4m3_values()):
        d = (abs(Fraction(float(v)) - t), b % 2)
        if best is None or d < best[0]:
            best = (d, Fraction(float(v)))
    return best[1] * g


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_quantize_matches_exact_rationals(fmt):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((6, 64)) * np.exp2(rng.integers(-20, 20, (6, 1)))
    x[1, 5] *= 50
    x[2] = 0
    x[3, 16:32] = 0
    x = O.to_bf16(np.where(x == 0, 1e-30, x)) * (x != 0)
    codes, scales, rows = O.quantize(x, fmt)
    got = O.values(codes, scales, rows, fmt)
    b = O.BLOCK[fmt]
    for r in range(len(x)):
        for h in range(64 // b):
            s = _exact_scale(x[r, h * b:(h + 1) * b], x[r], fmt)
            for k in range(h * b, (h + 1) * b):
                if s == 0:
                    assert got[r, k] == 0
                    continue
                v = abs(Fraction(float(x[r, k]))) / s
                i = min(range(8), key=lambda i: (abs(Fraction(float(O.LEVELS[i])) - min(v, 6)), i % 2))
                want = Fraction(float(O.LEVELS[i])) * s * (-1 if x[r, k] < 0 else 1)
                assert Fraction(float(got[r, k])) == want


def test_nonfinite_blocks():
    x = np.ones((1, 96))
    x[0, 3], x[0, 70] = np.nan, np.inf
    for fmt in O.BLOCK:
        codes, scales, rows = O.quantize(x, fmt)
        v = O.values(codes, scales, rows, fmt)
        b = O.BLOCK[fmt]
        assert np.isnan(v[0, :b]).all() and np.isnan(v[0, 70 // b * b:][:b]).all()
        assert np.isfinite(v[0, b:64]).all()


def test_layout_by_hand():
    # mxfp4, 2 x 64: 64 code bytes padded to 128, one chunk of 1024
    codes = (np.arange(128).reshape(2, 64) % 16).astype(np.uint8)
    scales = np.array([[1, 2], [3, 4]], np.uint8)
    out, known = O.pack(codes, scales, np.ones(2), "mxfp4")
    assert out.size == 128 + 1024 == O.packed_bytes(2, 64, "mxfp4")
    assert list(out[:3]) == [0x10, 0x32, 0x54] and out[32] == 0x10
    assert list(out[128:132]) == [1, 2, 0, 0] and list(out[144:148]) == [3, 4, 0, 0]
    assert known[:64].all() and not known[64:128].any() and known[128:].all()
    # row 33 (second column of lanes), scale 5 (second block) of nvfp4: chunk byte 512 + 16 + 4 + 1
    codes = np.zeros((40, 96), np.uint8)
    scales = np.zeros((40, 6), np.uint8)
    scales[33, 5] = 9
    out, _ = O.pack(codes, scales, np.full(40, 2.0, np.float32), "nvfp4")
    at = 1920 + 512 + 16 * 1 + 4 * 1 + 1
    assert out[at] == 9 and out[1920:1920 + 2048].sum() == 9
    assert out.size == 1920 + 2048 + 256
    assert out[1920 + 2048:1920 + 2048 + 160].view(np.float32).tolist() == [2.0] * 40


def test_route_by_hand():
    z = np.log(np.array([[1.0, 4.0, 2.0, 1.0]]))
    ids, w = O.route(z, 2)
    assert ids.tolist() == [[1, 2]] and np.allclose(w, [[0.5, 0.25]])
    ids, w = O.route(z, 3, renormalize=True, scale=2.0)
    assert ids.tolist() == [[1, 2, 0]] and np.allclose(w, [[8 / 7, 4 / 7, 2 / 7]])
    # the bias selects, the score weighs
    ids, w = O.route(z, 2, bias=np.array([0.9, 0, 0, 0.95]))
    assert ids.tolist() == [[3, 0]] and np.allclose(w, [[0.125, 0.125]])
    # groups {0,1} {2,3}: the first has the best expert
    ids, _ = O.route(z, 2, groups=2, top_groups=1)
    assert ids.tolist() == [[1, 0]]
    # nothing available
    ids, w = O.route(np.full((1, 4), -np.inf), 2, renormalize=True)
    assert ids.tolist() == [[0, 1]] and (w == 0).all()
    # one available of two chosen
    ids, w = O.route(np.array([[-np.inf, -np.inf, 0.0, -np.inf]]), 2)
    assert ids.tolist() == [[2, 0]] and w.tolist() == [[1.0, 0.0]]
