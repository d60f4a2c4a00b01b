"""fp64 oracle of the 4-bit weight format: E2M1 codes with one power-of-two
scale per 32 columns of a row, written from the field definitions.

A code is sign (bit 3), two exponent bits (bias 1) and one mantissa bit:
exponent 0 is m / 2, else (1 + m / 2) 2^(e - 1).  A scale byte b is 2^(b - 127)."""
from __future__ import annotations

import numpy as np

GROUP = 32


def e2m1_value(code: int) -> float:
    e, m = (code >> 1) & 3, code & 1
    mag = m / 2 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1)
    return -mag if code & 8 else mag


VALUES = np.array([e2m1_value(c) for c in range(16)])


def encode_rne(x: np.ndarray) -> np.ndarray:
    """Nearest code of each |x| <= 6, a tie to the even code, the sign kept."""
    x = np.asarray(x, np.float64)
    dist = np.abs(np.abs(x)[..., None] - VALUES[:8])
    near = dist == dist.min(axis=-1, keepdims=True)                # one code, or two neighbours
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(near.sum(axis=-1) > 1, even.argmax(axis=-1), near.argmax(axis=-1))
    return (code | np.signbit(x).astype(np.int64) << 3).astype(np.uint8)


def scale_exp(amax: float) -> int:
    """The first k from -126 up with amax <= 6 * 2^k; 0 for amax == 0."""
    if amax == 0.0:
        return 0
    k = -126
    while amax > 6.0 * 2.0 ** k:
        k += 1
    return k


def quantize_groups(x: np.ndarray):
    """(q [rows, cols / 2], scale [rows, cols / 32]) uint8 of x [rows, cols]; a
    group with an infinity or a NaN: codes 0 and scale 255 (NaN)."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    grp = x.reshape(rows, cols // GROUP, GROUP)
    finite = np.isfinite(grp).all(axis=2)
    grp = np.where(finite[..., None], grp, 0.0)
    k = np.vectorize(scale_exp, otypes=[np.int64])(np.abs(grp).max(axis=2))
    code = encode_rne(grp / np.ldexp(1.0, k)[..., None]).reshape(rows, cols // 2, 2)
    return (code[..., 0] | code[..., 1] << 4).astype(np.uint8), np.where(finite, k + 127, 255).astype(np.uint8)


def dequantize_groups(q: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """fp64 values [rows, cols]."""
    code = np.stack([q & 15, q >> 4], axis=-1).reshape(q.shape[0], -1)
    sc = np.where(scale == 255, np.nan, np.ldexp(1.0, scale.astype(np.int64) - 127))
    return VALUES[code] * np.repeat(sc, GROUP, axis=1)
