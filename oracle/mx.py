"""Reference of the microscaled (MX) operators in numpy and fp64 -- TEST INFRASTRUCTURE.

Only tests import this module; it shares no code with the CUDA library.  Elements are found
by search in the sorted list of representable values, scales by search over powers of two,
so nothing here mirrors the kernels' bit arithmetic.
"""

from __future__ import annotations

import numpy as np
from scipy.special import ndtr

BLOCK = 32
BLOCK_BYTES = {"e2m1": 16, "e4m3": 32}
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# codes 0..126: subnormals m * 2^-9, then (8 + m) * 2^(x - 10) for x = 1..15 (127 is NaN)
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)]
                + [(8 + m) * 2.0 ** (x - 10) for x in range(1, 16) for m in range(8)][:-1])
LEVELS = {"e2m1": E2M1, "e4m3": E4M3}
POWERS = 2.0 ** np.arange(-127, 128)


def scale_index(rows: int, blocks: int):
    """Byte offsets of the scales of every (row, block)."""
    r = np.arange(rows)[:, None]
    b = np.arange(blocks)[None, :]
    tiles_x = -(-blocks // 4)
    return ((r // 128) * tiles_x + b // 4) * 512 + (r % 32) * 16 + ((r % 128) // 32) * 4 + b % 4


def scale_bytes(rows: int, cols: int) -> int:
    blocks = -(-cols // BLOCK)
    return -(-rows // 128) * -(-blocks // 4) * 512


def quantize(x: np.ndarray, fmt: str):
    """(codes as uint8 rows x padded columns, scale bytes rows x blocks) of fp64 values x."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    pad = np.zeros((rows, blocks * BLOCK))
    pad[:, :cols] = x
    levels = LEVELS[fmt]
    blk = pad.reshape(rows, blocks, BLOCK)
    bad = ~np.isfinite(blk).all(axis=2)
    amax = np.abs(np.where(np.isfinite(blk), blk, 0)).max(axis=2)
    if fmt == "e2m1":  # the largest power with 4 * power <= amax
        e = np.searchsorted(4 * POWERS, amax, side="right") - 1
    else:  # the smallest power with amax <= 448 * power
        e = np.searchsorted(448 * POWERS, amax, side="left")
    e = np.clip(e, 0, 254)
    e[amax == 0] = 0
    a = np.abs(np.where(np.isfinite(blk), blk, 0)) / POWERS[e][:, :, None]
    hi = np.minimum(np.searchsorted(levels, a), len(levels) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - levels[lo], levels[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(a >= levels[-1], len(levels) - 1, code)
    sign = np.signbit(blk)
    code = code + np.where(sign, 8 if fmt == "e2m1" else 128, 0)
    scale = np.where(bad, 255, e).astype(np.uint8)
    return code.astype(np.uint8).reshape(rows, -1), scale


def pack(codes: np.ndarray, fmt: str) -> np.ndarray:
    """Codes as the bytes of Q."""
    return codes if fmt == "e4m3" else (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(Q: np.ndarray, fmt: str) -> np.ndarray:
    if fmt == "e4m3":
        return Q
    out = np.empty((Q.shape[0], Q.shape[1] * 2), dtype=np.uint8)
    out[:, 0::2], out[:, 1::2] = Q & 15, Q >> 4
    return out


def tile_scales(scale: np.ndarray, fill: int = 0) -> np.ndarray:
    """Scale bytes (rows x blocks) as the buffer S; padding blocks 0, padding rows `fill`."""
    rows, blocks = scale.shape
    padded = np.zeros((rows, -(-blocks // 4) * 4), dtype=np.uint8)
    padded[:, :blocks] = scale
    S = np.full(scale_bytes(rows, blocks * BLOCK), fill, dtype=np.uint8)
    S[scale_index(rows, padded.shape[1])] = padded
    return S


def decode(codes: np.ndarray, scale: np.ndarray, fmt: str) -> np.ndarray:
    """fp64 values of codes (rows x padded columns) and scale bytes (rows x blocks)."""
    half = 8 if fmt == "e2m1" else 128
    mag = codes % half
    if fmt == "e2m1":
        v = E2M1[mag]
    else:
        v = np.append(E4M3, np.nan)[mag]
    s = np.append(POWERS, np.nan)[scale]
    return np.where(codes >= half, -v, v) * np.repeat(s, BLOCK, axis=1)


def activate(act: str, x: np.ndarray) -> np.ndarray:
    x = np.asarray(x, dtype=np.float64)
    if act == "none":
        return x
    if act == "relu":
        return np.maximum(x, 0)
    if act == "gelu":
        return x * ndtr(x)
    c, w = (0.0, 1.0) if act == "silu" else (0.044715, 2 * np.sqrt(2 / np.pi))
    return x / (1 + np.exp(-w * (x + c * x ** 3)))


def slope(act: str, x: np.ndarray) -> np.ndarray:
    """The derivative of activate."""
    x = np.asarray(x, dtype=np.float64)
    if act == "none":
        return np.ones_like(x)
    if act == "relu":
        return np.where(np.isnan(x), np.nan, (x > 0).astype(np.float64))
    if act == "gelu":
        return ndtr(x) + x * np.exp(-x * x / 2) / np.sqrt(2 * np.pi)
    c, w = (0.0, 1.0) if act == "silu" else (0.044715, 2 * np.sqrt(2 / np.pi))
    u = w * (x + c * x ** 3)
    s, r = 1 / (1 + np.exp(-u)), 1 / (1 + np.exp(u))
    return s + x * s * r * w * (1 + 3 * c * x * x)
