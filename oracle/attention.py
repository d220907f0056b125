"""float64 reference of the attention side of the block: head norms and
rotation with their gradients, the paged cache append and attention over the
paged cache.  Plain numpy, no code shared with the library."""
from __future__ import annotations

import math

import numpy as np


def angles(table, positions, rot):
    """cos and sin [T, rot/2] of every token's position; NaN outside the table."""
    table = np.asarray(table, dtype=np.float64)
    positions = np.asarray(positions, dtype=np.int64)
    ok = (positions >= 0) & (positions < len(table))
    rows = np.where(ok[:, None], table[np.where(ok, positions, 0)], np.nan)
    return rows[:, :rot // 2], rows[:, rot // 2:]


def pair_indices(rot, adjacent):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if adjacent else (i, i + rot // 2)


def rotate(x, c, s, rot, adjacent, transposed=False):
    """Rotation of the pairs of x [T, H, D] by the angles of each token."""
    y = np.array(x, dtype=np.float64)
    if rot == 0:
        return y
    a, b = pair_indices(rot, adjacent)
    sign = -1.0 if transposed else 1.0
    c, s = c[:, None, :], sign * s[:, None, :]
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return y


def norm_rope(x, w, table, positions, rot, adjacent=False, norm=True, eps=1e-6):
    x = np.asarray(x, dtype=np.float64)
    if norm:
        r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        x = x * r * (1.0 if w is None else np.asarray(w, dtype=np.float64))
    c, s = angles(table, positions, rot) if rot else (None, None)
    return rotate(x, c, s, rot, adjacent)


def norm_rope_backward(x, w, table, positions, gy, rot, adjacent=False, norm=True, eps=1e-6):
    """Gradients of x and of w (None without the norm) from that of the output."""
    gy = np.asarray(gy, dtype=np.float64)
    c, s = angles(table, positions, rot) if rot else (None, None)
    gn = rotate(gy, c, s, rot, adjacent, transposed=True)
    if not norm:
        return gn, None
    x = np.asarray(x, dtype=np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * r
    gw = (gn * xh).sum((0, 1))
    gh = gn * (1.0 if w is None else np.asarray(w, dtype=np.float64))
    return r * (gh - xh * (gh * xh).mean(-1, keepdims=True)), gw


def paged_append(cache, rows, slots):
    """The cache [n_pages, page_size, H, D] with rows [T, H, D] in their slots."""
    out = np.array(cache, dtype=np.float64)
    n, page = out.shape[:2]
    for t, slot in enumerate(np.asarray(slots, dtype=np.int64)):
        if 0 <= slot < n * page:
            out[slot // page, slot % page] = rows[t]
    return out


def paged_attention(q, k_cache, v_cache, q_start, kv_len, block_table, scale, causal=True,
                    window=0):
    """out [T, Hq, D] and lse [T, Hq]; rows of no sequence are NaN.  Also, per
    row and head, the scales of its rounding bounds: a weighted mean of |v|
    [T, Hq, D] and the largest scale * sum |q| |k| over the keys it sees."""
    q = np.asarray(q, dtype=np.float64)
    T, hq, D = q.shape
    hkv, page = k_cache.shape[2], k_cache.shape[1]
    out, lse = np.full((T, hq, D), np.nan), np.full((T, hq), np.nan)
    mag, smax = np.zeros((T, hq, D)), np.zeros((T, hq))
    for b in range(len(kv_len)):
        r0, r1, n = int(q_start[b]), int(q_start[b + 1]), int(kv_len[b])
        j = np.arange(n)
        pages = np.asarray(block_table)[b][j // page] if n else np.zeros(0, dtype=np.int64)
        pos = n - (r1 - r0) + np.arange(r1 - r0)
        seen = np.ones((r1 - r0, n), dtype=bool)
        if causal:
            seen &= j[None, :] <= pos[:, None]
        if window > 0:
            seen &= j[None, :] > pos[:, None] - window
        # keys that no row sees are not looked at
        live = seen.any(0)
        j, pages, seen = j[live], pages[live], seen[:, live]
        for h in range(hq):
            k = np.asarray(k_cache[pages, j % page, h // (hq // hkv)], dtype=np.float64)
            v = np.asarray(v_cache[pages, j % page, h // (hq // hkv)], dtype=np.float64)
            qs = q[r0:r1, h]
            with np.errstate(invalid="ignore"):
                z = np.where(seen, scale * (qs @ k.T), -math.inf)
            for i in range(r1 - r0):
                keys = seen[i]
                if not keys.any():
                    out[r0 + i, h], lse[r0 + i, h] = 0.0, -math.inf
                    continue
                zi = z[i, keys]
                top = zi.max()
                e = np.exp(zi - top)
                p = e / e.sum()
                out[r0 + i, h] = p @ v[keys]
                lse[r0 + i, h] = top + math.log(e.sum())
                mag[r0 + i, h] = p @ np.abs(v[keys])
                smax[r0 + i, h] = abs(scale) * (np.abs(k[keys]) @ np.abs(qs[i])).max()
    return out, lse, mag, smax
