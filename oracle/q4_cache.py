"""The 4-bit cache rows on the CPU: quantisation, packing and what rows stand for.

Written from the format's definition in ``include/pagedattn.h`` with numpy;
shares no code with the GPU path.  Every step of the quantisation is one fp32
operation, as the definition says, so the bytes are exactly determined.
"""
from __future__ import annotations

import numpy as np

MAX = np.float32(16384.0)


def row_bytes(hkv: int, hd: int, gs: int) -> int:
    par = hkv * (hd // gs) * 4
    return hkv * hd // 2 + -(-par // 16) * 16


def quantise(x, gs: int):
    """fp32 x [n, Hkv, hd] -> codes uint8 [n, Hkv, hd], s and c float16 [n, Hkv, hd // gs]."""
    x = np.asarray(x, dtype=np.float32)
    n, hkv, hd = x.shape
    g = x.reshape(n, hkv, hd // gs, gs)
    good = np.isfinite(g).all(-1)
    g = np.clip(np.where(good[..., None], g, np.float32(0)), -MAX, MAX)
    mn, mx = g.min(-1), g.max(-1)
    s = ((mx - mn) * np.float32(1.0 / 15.0)).astype(np.float16)
    c = (mn - np.float32(16) * s.astype(np.float32)).astype(np.float16)
    sf, cf = s.astype(np.float32)[..., None], c.astype(np.float32)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        r = np.where(sf > 0, np.float32(1) / sf, np.float32(0)).astype(np.float32)
        t = np.clip(np.rint((g - cf) * r), 16, 31)
    u = np.where(sf > 0, t - 16, 0).astype(np.uint8)
    u = np.where(good[..., None], u, 0)
    return (u.reshape(n, hkv, hd), np.where(good, s, np.float16(0)),
            np.where(good, c, np.float16(np.nan)))


def values(u, s, c, gs: int):
    """float64 values [n, Hkv, hd] of codes and parameters."""
    with np.errstate(invalid="ignore"):     # parameters of unwritten rows may be any NaN
        s = np.repeat(np.asarray(s, dtype=np.float64), gs, axis=-1)
        c = np.repeat(np.asarray(c, dtype=np.float64), gs, axis=-1)
        return s * (16.0 + np.asarray(u, dtype=np.float64)) + c


def _move(part, slots):
    """Exchange 16-byte pieces j and j ^ (slot mod pieces) inside blocks of up to 8 pieces (its own inverse)."""
    n, size = part.shape
    pieces = min(8, size // 16)
    p = part.reshape(n, size // (16 * pieces), pieces, 16)
    j = np.arange(pieces)[None, :] ^ (np.asarray(slots, dtype=np.int64)[:, None] % pieces)
    return np.take_along_axis(p, j[:, None, :, None], axis=2).reshape(n, size)


def pack_rows(u, s, c, slots):
    """Cache rows uint8 [n, row bytes] for the given slots (padding bytes 0)."""
    n, hkv, hd = u.shape
    q = np.asarray(u, dtype=np.uint16).reshape(n, hkv * hd // 4, 4)
    half = ((q[..., 0] << 6) | (q[..., 2] << 2) | (q[..., 3] << 10) | ((q[..., 1] & 3) << 14) | (q[..., 1] >> 2))
    codes = half.astype("<u2").view(np.uint8).reshape(n, hkv * hd // 2)
    words = np.stack([np.asarray(s, np.float16), np.asarray(c, np.float16)], -1).astype("<f2")
    par = words.reshape(n, -1).view(np.uint8).reshape(n, -1)
    par = np.pad(par, ((0, 0), (0, -par.shape[1] % 16)))
    return np.concatenate([_move(codes, slots), _move(par, slots)], axis=1)


def unpack_rows(rows, slots, hkv: int, hd: int, gs: int):
    """Codes, s and c of cache rows."""
    n, nc = rows.shape[0], hkv * hd // 2
    half = np.ascontiguousarray(_move(rows[:, :nc], slots)).view("<u2").reshape(n, hkv * hd // 4)
    u = np.stack([(half >> 6) & 15, (half >> 14) | ((half & 3) << 2), (half >> 2) & 15, (half >> 10) & 15], -1)
    par = np.ascontiguousarray(_move(rows[:, nc:], slots)).view("<f2").reshape(n, -1)[:, : hkv * (hd // gs) * 2]
    par = par.reshape(n, hkv, hd // gs, 2)
    return u.reshape(n, hkv, hd).astype(np.uint8), par[..., 0], par[..., 1]


def row_values(rows, slots, hkv: int, hd: int, gs: int):
    """float64 values [n, Hkv, hd] of cache rows."""
    return values(*unpack_rows(rows, slots, hkv, hd, gs), gs)
