"""Microscaled 4-bit formats in 64 bits (numpy): quantise, the values stored,
packing and the scale tiles.  Test infrastructure; every step follows the
definition in include/qlora.h and none is shared with the library."""
from __future__ import annotations

import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = {"mxfp4": 32, "nvfp4": 16}
NAN_BYTE = {"mxfp4": 255, "nvfp4": 0x7F}


def nearest_code(v: np.ndarray) -> np.ndarray:
    """Code 0..7 of the level nearest to v >= 0, ties to the even code."""
    d = np.abs(v[..., None] - LEVELS)
    best = d.min(axis=-1, keepdims=True)
    hit = d == best                              # one level, or two on a tie
    first = hit.argmax(axis=-1)
    last = 7 - hit[..., ::-1].argmax(axis=-1)
    return np.where(first % 2 == 0, first, last).astype(np.uint8)


def e4m3_levels() -> np.ndarray:
    """The 127 non-negative finite E4M3 values, by byte."""
    b = np.arange(127)
    e, m = b >> 3, b & 7
    return np.where(e == 0, m / 512.0, (1 + m / 8.0) * 2.0 ** (e - 7.0))


def nearest_e4m3(v: np.ndarray) -> np.ndarray:
    lv = e4m3_levels()
    hi = np.clip(np.searchsorted(lv, v), 1, 126)
    lo = hi - 1
    dl, dh = v - lv[lo], lv[hi] - v
    take_hi = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(take_hi, hi, lo).astype(np.uint8)


def global_scale(amax: float) -> float:
    if amax == 0:
        return 1.0
    e = -126
    while amax > 2688.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def quantize(x: np.ndarray, fmt: str, per_row: bool = False):
    """x float64 [rows, cols] -> (codes [rows, cols], scale bytes [rows, blocks], g [1] or [rows] or None)."""
    rows, cols = x.shape
    blk = BLOCK[fmt]
    nb = -(-cols // blk)
    b = np.concatenate([x, np.zeros((rows, nb * blk - cols))], axis=1).reshape(rows, nb, blk)
    finite = np.isfinite(b)
    bad = ~finite.all(axis=2)
    mag = np.where(finite, np.abs(b), 0.0)
    amax = mag.max(axis=2)
    if fmt == "mxfp4":
        with np.errstate(divide="ignore"):
            e = np.where(amax > 0, np.frexp(amax)[1] - 1 - 2, -127).clip(-127)
        sb, g = (e + 127).astype(np.uint8), None
        step = 2.0 ** e
    else:
        tops = amax.max(axis=1) if per_row else np.array([amax.max()])
        g = np.array([global_scale(t) for t in tops])
        gr = np.broadcast_to(g, (rows,))[:, None]
        sb = nearest_e4m3(amax / gr / 6.0)
        step = e4m3_levels()[sb] * gr
    with np.errstate(divide="ignore", invalid="ignore"):
        v = np.where(step[..., None] > 0, mag / step[..., None], 0.0)
    codes = nearest_code(v)
    codes = codes | (np.signbit(b).astype(np.uint8) << 3)
    if fmt == "nvfp4":
        codes = np.where(sb[..., None] == 0, 0, codes)
    codes = np.where(bad[..., None], 0, codes).astype(np.uint8)
    sb = np.where(bad, NAN_BYTE[fmt], sb).astype(np.uint8)
    return codes.reshape(rows, nb * blk)[:, :cols], sb, g


def values(codes: np.ndarray, sb: np.ndarray, g, fmt: str) -> np.ndarray:
    rows, cols = codes.shape
    blk = BLOCK[fmt]
    if fmt == "mxfp4":
        s = np.where(sb == 255, np.nan, 2.0 ** (sb.astype(np.float64) - 127))
    else:
        s = np.append(e4m3_levels(), np.nan)[np.minimum(sb, 127)]
        s = s * np.broadcast_to(g, (rows,))[:, None]
    s = np.repeat(s, blk, axis=1)[:, :cols]
    return LEVELS[codes & 7] * np.where(codes & 8, -1.0, 1.0) * s


def pack(codes: np.ndarray) -> np.ndarray:
    """[rows, cols] codes -> bytes [rows, 16 * ceil(cols / 32)], the earlier code in the low bits."""
    rows, cols = codes.shape
    p = np.zeros((rows, -(-cols // 32) * 32), np.uint8)
    p[:, :cols] = codes
    return p[:, 0::2] | (p[:, 1::2] << 4)


def tile_scales(sb: np.ndarray) -> np.ndarray:
    """[rows, blocks] scale bytes -> the tile order, one byte at a time; absent ones 0."""
    rows, nb = sb.shape
    kt = -(-nb // 4)
    out = np.zeros((-(-rows // 128)) * kt * 512, np.uint8)
    r, b = np.meshgrid(np.arange(rows), np.arange(nb), indexing="ij")
    out[(r // 128 * kt + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4] = sb
    return out


def round_trip(x: np.ndarray, fmt: str, per_row: bool = False) -> np.ndarray:
    return values(*quantize(x, fmt, per_row), fmt)
