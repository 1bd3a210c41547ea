"""CPU oracle of the microscaled 4-bit format, its product, the routing to
experts and the experts' layer.

TEST INFRASTRUCTURE ONLY, in plain numpy and fp64, written from the
definitions in ``include/lutq.h``; it shares no code with the CUDA library.
Quantization decisions on bf16 and fp16 inputs are those of exact arithmetic:
the quantities compared (m / 6 / g, x / (s g)) have far fewer bits than fp64.
"""
from __future__ import annotations

from typing import Optional, Tuple

import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = {"mxfp4": 32, "nvfp4": 16}
NAN_SCALE = {"mxfp4": 0xFF, "nvfp4": 0x7F}


def _floor_log2(v: np.ndarray) -> np.ndarray:
    """floor(log2 v) for v > 0 (exact, from the binary exponent)."""
    return np.frexp(v)[1] - 1


def e4m3_values() -> np.ndarray:
    """The 127 finite non-negative E4M3 values in order (byte 0..126)."""
    b = np.arange(127)
    e, m = b >> 3, b & 7
    return np.where(e > 0, np.exp2(e - 7.0) * (1 + m / 8.0), m / 512.0)


def _nearest_even(v: np.ndarray, table: np.ndarray) -> np.ndarray:
    """Index of the value of the ascending table nearest to v >= 0, ties to the
    even index; values beyond the table take its last entry."""
    mid = (table[:-1] + table[1:]) / 2
    lo = np.searchsorted(mid, v, side="left")       # midpoints below v
    hi = np.searchsorted(mid, v, side="right")      # midpoints at or below v
    return np.where((hi > lo) & (lo % 2 == 1), hi, lo)


def quantize(x: np.ndarray, fmt: str) -> Tuple[np.ndarray, np.ndarray, np.ndarray]:
    """x [..., K] -> codes uint8 [..., K] (0..15), scale bytes [..., K / block]
    and row scales fp32 [...] (1 for mxfp4)."""
    x = np.asarray(x, np.float64)
    b = BLOCK[fmt]
    xb = x.reshape(*x.shape[:-1], -1, b)
    finite = np.isfinite(xb)
    bad = ~finite.all(-1)
    mag = np.where(finite, np.abs(xb), 0.0)
    m = mag.max(-1)
    if fmt == "mxfp4":
        e = np.where(m > 0, _floor_log2(np.where(m > 0, m, 1.0)) - 2, -127)
        e = np.maximum(e, -127)
        scales = (e + 127).astype(np.uint8)
        s = np.exp2(e.astype(np.float64))
        rows = np.ones(x.shape[:-1])
    else:
        r = mag.max((-1, -2))
        g = np.where(r > 0, _floor_log2(np.where(r > 0, r, 1.0)) - 10, 0)
        rows = np.exp2(np.maximum(g, -126).astype(np.float64))
        table = e4m3_values()
        scales = _nearest_even(m / 6.0 / rows[..., None], table).astype(np.uint8)
        s = table[scales] * rows[..., None]
    s = s[..., None]
    q = _nearest_even(np.where(s > 0, mag / np.where(s > 0, s, 1.0), 0.0), LEVELS)
    codes = np.where(np.signbit(xb), 8, 0) + q
    codes = np.where(bad[..., None], 0, codes).astype(np.uint8)
    scales = np.where(bad, NAN_SCALE[fmt], scales).astype(np.uint8)
    return codes.reshape(x.shape), scales, rows.astype(np.float32)


def values(codes, scales, rows, fmt: str) -> np.ndarray:
    """The fp64 values that codes [..., K], scale bytes and row scales stand for."""
    lv = np.concatenate([LEVELS, -LEVELS])[codes]
    if fmt == "mxfp4":
        s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    else:
        table = np.concatenate([e4m3_values(), [np.nan]])
        s = np.where(scales >> 7, -1.0, 1.0) * table[scales & 127]
        s = s * np.asarray(rows, np.float64)[..., None]
    return (lv.reshape(*lv.shape[:-1], -1, BLOCK[fmt]) * s[..., None]).reshape(lv.shape)


def packed_bytes(n: int, k: int, fmt: str) -> int:
    up = lambda v, m: -(-v // m) * m  # noqa: E731
    chunk = 1024 if fmt == "mxfp4" else 2048
    return (up(n * k // 2, 128) + (up(n, 128) // 128) * (up(k, 256) // 256) * chunk
            + (up(4 * n, 128) if fmt == "nvfp4" else 0))


def pack(codes, scales, rows, fmt: str) -> Tuple[np.ndarray, np.ndarray]:
    """The packed bytes of one matrix and a mask of those that are specified."""
    n, k = codes.shape
    out = np.zeros(packed_bytes(n, k, fmt), np.uint8)
    known = np.ones(out.size, bool)
    pair = codes[:, 0::2] | (codes[:, 1::2] << 4)
    out[:pair.size] = pair.ravel()
    base = -(-pair.size // 128) * 128
    known[pair.size:base] = False
    chunk = 1024 if fmt == "mxfp4" else 2048
    chunks = -(-k // 256)
    r, h = np.meshgrid(np.arange(n), np.arange(scales.shape[1]), indexing="ij")
    per = 256 // BLOCK[fmt]
    at = (base + ((r // 128) * chunks + h // per) * chunk + (h % per) // 4 * 512
          + 16 * (r % 32) + 4 * ((r % 128) // 32) + h % 4)
    out[at.ravel()] = scales.ravel()
    if fmt == "nvfp4":
        end = base + -(-n // 128) * chunks * chunk
        out[end:end + 4 * n] = np.asarray(rows, np.float32).view(np.uint8)
        known[end + 4 * n:] = False
    return out, known


def product(xv: np.ndarray, wv: np.ndarray) -> Tuple[np.ndarray, np.ndarray]:
    """x w^T and the sum of the products' magnitudes, in fp64."""
    return xv @ wv.T, np.abs(xv) @ np.abs(wv).T


def route(z, top_k: int, score: str = "softmax", bias: Optional[np.ndarray] = None,
          groups: int = 1, top_groups: int = 1, group_best: int = 1, renormalize: bool = False,
          scale: float = 1.0) -> Tuple[np.ndarray, np.ndarray]:
    """ids and weights (fp64) of every row of logits z, token by token."""
    z = np.asarray(z, np.float64)
    ids = np.zeros((len(z), top_k), np.int32)
    weights = np.zeros((len(z), top_k))
    for t, row in enumerate(z):
        row = np.where(np.isnan(row), -np.inf, row)
        there = row > -np.inf
        p = np.zeros(len(row))
        if score == "softmax":
            if there.any():
                top = row.max()
                with np.errstate(invalid="ignore"):
                    e = np.where(row == top, 1.0, np.exp(row - top))
                e = np.where(there, e, 0.0)
                p = e / e.sum()
        else:
            p = np.where(there, 1.0 / (1.0 + np.exp(-np.where(there, row, 0.0))), 0.0)
        c = p + (0.0 if bias is None else np.asarray(bias, np.float64))
        c = np.where(there, c, -np.inf)
        if groups > 1:
            per = len(row) // groups
            gs = []
            for g in range(groups):
                best = sorted((v for v in c[g * per:(g + 1) * per] if v > -np.inf), reverse=True)
                gs.append(sum(best[:group_best]) if best else -np.inf)
            kept = sorted(range(groups), key=lambda g: (-gs[g], g))[:top_groups]
            c = np.where(np.isin(np.arange(len(row)) // per, kept), c, -np.inf)
        order = sorted(range(len(row)), key=lambda e: (-c[e], e))[:top_k]
        w = np.array([p[e] if c[e] > -np.inf else 0.0 for e in order])
        if renormalize:
            w = w / w.sum() if w.sum() > 0 else w
        ids[t], weights[t] = order, w * scale
    return ids, weights


def to_bf16(v: np.ndarray) -> np.ndarray:
    """fp64 -> the nearest bf16 (ties to even), as fp64; for |v| within the normal range."""
    m, e = np.frexp(v)
    return np.ldexp(np.round(m * 256.0), e - 8)


def experts(xv, ids, weights, gate, up, down, fmt: str) -> np.ndarray:
    """y of the layer: xv [T, D] the values of quantized x; gate, up [E, F, D]
    and down [E, D, F] values."""
    y = np.zeros(xv.shape)
    for t in range(len(xv)):
        for j, e in enumerate(ids[t]):
            if not 0 <= e < len(gate):
                continue
            g, u = gate[e] @ xv[t], up[e] @ xv[t]
            h = to_bf16(g / (1.0 + np.exp(-g)) * u)
            y[t] += weights[t, j] * (down[e] @ values(*quantize(h, fmt), fmt))
    return y
