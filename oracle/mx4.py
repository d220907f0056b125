"""float64 reference of the 4-bit form of cached keys and values (OCP MX FP4 in blocks of 32
elements of a head).  Plain numpy, no code shared with the library."""
from __future__ import annotations

import numpy as np

BLOCK = 32
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def blocks(dim):
    return -(-dim // BLOCK)


def encode(x):
    """Codes uint8 [..., dim / 2] and scale bytes uint8 [..., blocks] of x [..., dim]."""
    x = np.asarray(x, dtype=np.float64)
    dim = x.shape[-1]
    code = np.zeros(x.shape, dtype=np.uint8)
    scale = np.zeros(x.shape[:-1] + (blocks(dim),), dtype=np.uint8)
    for b in range(blocks(dim)):
        part = x[..., b * BLOCK:(b + 1) * BLOCK]
        top = np.abs(part).max(-1)
        fine = np.isfinite(top)
        e = np.full(top.shape, -124)
        while True:
            more = fine & (e < 125) & (top >= 7.0 * np.exp2(e.astype(np.float64)))
            if not more.any():
                break
            e = e + more
        m = np.abs(np.where(fine[..., None], part, 0.0)) / np.exp2(e.astype(np.float64))[..., None]
        # the nearest magnitude; of two as near the one with the even code
        c = np.zeros(m.shape, dtype=np.uint8)
        for i in range(7):
            mid = (MAGNITUDES[i] + MAGNITUDES[i + 1]) / 2
            c += (m > mid) | ((m == mid) & (i % 2 == 1))
        code[..., b * BLOCK:(b + 1) * BLOCK] = c + 8 * (np.signbit(part) & fine[..., None])
        scale[..., b] = np.where(fine, e + 127, 255)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale


def decode(codes, scales):
    """The values of codes [..., dim / 2] and their scale bytes."""
    code = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    x = np.where(code & 8, -1.0, 1.0) * MAGNITUDES[code & 7]
    s = scales.astype(np.float64)
    factor = np.where(scales >= 253, np.nan, np.exp2(s - 127))
    return x * np.repeat(factor, BLOCK, -1)[..., :x.shape[-1]]
