"""Oracle of the 4-bit caches and of windowed attention: numpy float64, from
the definitions alone (test infrastructure; shares no code with the CUDA
path).

The 4-bit format: per block of 16 columns a scale byte (5 exponent bits, bias
15, over 3 mantissa bits) and per column an E2M1 code; the scale is the
representable number nearest to amax / 6 (ties to the even byte) and at most
10240, the code the representable number nearest to x / scale (ties to the
even code).
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
MAX_SCALE_BYTE = 226  # 10240


def scale_value(byte) -> np.ndarray:
    b = np.asarray(byte).astype(np.int64)
    e, m = b >> 3, (b & 7).astype(np.float64)
    return np.where(e > 0, (1 + m / 8) * np.exp2(np.where(e > 0, e, 1) - 15.0), m / 8 * 2.0 ** -14)


_SCALES = scale_value(np.arange(MAX_SCALE_BYTE + 1))


def _nearest_even(x, grid) -> np.ndarray:
    """Index of the nearest entry of an ascending grid, ties to the even index;
    values past the last entry take it."""
    hi = np.clip(np.searchsorted(grid, x), 0, len(grid) - 1)
    lo = np.clip(hi - 1, 0, None)
    dl, dh = np.abs(x - grid[lo]), np.abs(grid[hi] - x)
    return np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


def quantise(x) -> tuple:
    """x [..., w] -> (codes [..., w] 0..15, scale bytes [..., w / 16])."""
    x = np.asarray(x, dtype=np.float64)
    blk = x.reshape(*x.shape[:-1], -1, 16)
    byte = _nearest_even(np.abs(blk).max(-1) / 6, _SCALES)
    s = _SCALES[byte][..., None]
    mag = _nearest_even(np.abs(blk) / np.where(s > 0, s, 1.0), E2M1)
    mag = np.where(s > 0, mag, 0)
    code = mag + 8 * ((blk < 0) & (mag > 0))
    return code.reshape(x.shape), byte


def values(codes, scales) -> np.ndarray:
    codes = np.asarray(codes)
    v = E2M1[codes & 7] * np.repeat(scale_value(scales), 16, axis=-1)
    return np.where(codes & 8, -v, v)


def round4(x) -> np.ndarray:
    """What a row reads back as."""
    return values(*quantise(x))


def pack_tile(x) -> np.ndarray:
    """One tile [S][w] of floats -> its bytes."""
    codes, scales = quantise(x)
    by = codes[:, 0::2] | (codes[:, 1::2] << 4)
    return np.concatenate([by.reshape(-1), scales.reshape(-1)]).astype(np.uint8)


def unpack_tile(t, S: int, w: int) -> np.ndarray:
    """Bytes of one tile -> values [S][w]."""
    t = np.asarray(t).astype(np.int64)
    by, sc = t[:S * w // 2].reshape(S, w // 2), t[S * w // 2:].reshape(S, w // 16)
    codes = np.stack([by & 15, by >> 4], -1).reshape(S, w)
    return values(codes, sc)


def mix(q, K, Z, see) -> np.ndarray:
    """q [n][d], K [T][d], Z [T][r], see [n][T] -> softmax(q K^T / sqrt d) Z over
    the tokens a row sees; rows that see nothing are zero."""
    out = np.zeros((q.shape[0], Z.shape[1]))
    for i in range(q.shape[0]):
        t = np.flatnonzero(see[i])
        if len(t):
            s = K[t] @ q[i] / np.sqrt(q.shape[1])
            p = np.exp(s - s.max())
            out[i] = p @ Z[t] / p.sum()
    return out


def window_mask(L: int, n: int, window: int, sink: int) -> np.ndarray:
    """[n][L]: which tokens the last n of L tokens see (rows at negative
    positions see nothing)."""
    p = np.arange(L - n, L)[:, None]
    t = np.arange(L)[None]
    see = t <= p
    if window:
        see &= (t > p - window) | (t < sink)
    return see
