"""Reference of the 8-bit checkpoint form in numpy (no GPU): blocks of 32
columns, scale byte b = the least with max|x| <= limit * 2^(b-127), codes
x / scale rounded to nearest even (int8, limit 127; E4M3, limit 448)."""
from __future__ import annotations

import math

import numpy as np

from tests.fp8_ref import e4m3_table

I8, E4M3 = 1, 2
LIMIT = {I8: 127.0, E4M3: 448.0}


def _scale_byte(a: float, limit: float) -> int:
    """By the definition: try the bytes around the logarithm."""
    if not math.isfinite(a):
        return 255
    if a == 0:
        return 0
    b = max(0, int(math.floor(math.log2(a / limit))) + 127 - 2)
    while a > limit * 2.0 ** (b - 127):
        b += 1
    return b


def _round_e4m3(q: np.ndarray) -> np.ndarray:
    """Nearest E4M3 value (ties to even) of |q| <= 448: a multiple of the step at its exponent."""
    e = np.floor(np.log2(np.maximum(np.abs(q), 2.0 ** -30)))
    e = np.where(np.abs(q) < 2.0 ** e, e - 1, np.where(np.abs(q) >= 2.0 ** (e + 1), e + 1, e))
    step = 2.0 ** (np.maximum(e, -6.0) - 3.0)
    return np.rint(q / step) * step


def scales_of(x: np.ndarray, fmt: int) -> np.ndarray:
    """Scale bytes [T, ceil(n/32)] of x [T, n]."""
    T, n = x.shape
    nb = -(-n // 32)
    out = np.zeros((T, nb), np.uint8)
    for k in range(nb):
        blk = np.abs(x[:, 32 * k:32 * k + 32]).astype(np.float64)
        a = np.where(np.isnan(blk).any(axis=1), np.inf, np.max(np.nan_to_num(blk, nan=0.0, posinf=np.inf), axis=1))
        out[:, k] = [_scale_byte(float(v), LIMIT[fmt]) for v in a]
    return out


def values_of(x: np.ndarray, fmt: int) -> np.ndarray:
    """What the packed form of x stands for (float64)."""
    T, n = x.shape
    b = np.repeat(scales_of(x, fmt).astype(np.float64), 32, axis=1)[:, :n]
    s = 2.0 ** (b - 127)
    with np.errstate(invalid="ignore"):
        q = x.astype(np.float64) / s
        q = np.rint(q) if fmt == I8 else _round_e4m3(np.where(b == 255, 0, q))
        return np.where(b == 255, np.nan, q * s)


def decode(codes: np.ndarray, scales: np.ndarray, fmt: int) -> np.ndarray:
    """float64 values of codes [T, n] with scale bytes [T, ceil(n/32)]."""
    n = codes.shape[1]
    b = np.repeat(scales.astype(np.float64), 32, axis=1)[:, :n]
    v = codes.view(np.int8).astype(np.float64) if fmt == I8 else e4m3_table()[codes].astype(np.float64)
    return np.where(b == 255, np.nan, v * 2.0 ** (b - 127))
