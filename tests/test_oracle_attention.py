"""The float64 reference of the attention side against independent forms:
loops over single elements, and differences for the gradients (CPU)."""
from __future__ import annotations

import math

import numpy as np
import pytest

from oracle import attention as A


def _table(rows, rot):
    f = 10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))
    a = np.arange(rows)[:, None] * f[None, :]
    return np.concatenate([np.cos(a), np.sin(a)], 1)


@pytest.mark.parametrize("adjacent", [False, True])
def test_rotation_is_a_complex_product(adjacent):
    rng = np.random.default_rng(0)
    x, rot, pos = rng.standard_normal((5, 3, 16)), 12, np.array([0, 3, 7, 1, 9])
    y = A.norm_rope(x, None, _table(10, rot), pos, rot, adjacent, norm=False)
    a, b = A.pair_indices(rot, adjacent)
    turn = np.exp(1j * pos[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot))[:, None, :]
    z = (x[..., a] + 1j * x[..., b]) * turn
    assert np.allclose(y[..., a], z.real) and np.allclose(y[..., b], z.imag)
    assert np.array_equal(y[..., rot:], x[..., rot:])


@pytest.mark.parametrize("rot,adjacent,norm", [(8, False, True), (4, True, True), (0, False, True),
                                               (8, True, False)])
def test_gradients_against_differences(rot, adjacent, norm):
    rng = np.random.default_rng(1)
    x, w, gy = rng.standard_normal((4, 3, 8)), rng.standard_normal(8), rng.standard_normal((4, 3, 8))
    pos, tab = np.array([5, 0, 2, 9]), _table(10, rot)

    def loss(x, w):
        return (A.norm_rope(x, w, tab, pos, rot, adjacent, norm, 1e-3) * gy).sum()

    gx, gw = A.norm_rope_backward(x, w, tab, pos, gy, rot, adjacent, norm, 1e-3)
    h = 1e-5
    for idx in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[idx] = h
        # a central difference errs by h^2 and by rounding / h
        assert abs((loss(x + d, w) - loss(x - d, w)) / (2 * h) - gx[idx]) < 1e-7
    if norm:
        for i in range(8):
            d = np.zeros_like(w)
            d[i] = h
            assert abs((loss(x, w + d) - loss(x, w - d)) / (2 * h) - gw[i]) < 1e-7
    else:
        assert gw is None


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 3), (False, 2)])
def test_attention_against_loops(causal, window):
    rng = np.random.default_rng(2)
    page, hq, hkv, D = 3, 4, 2, 5
    q_start, kv_len = [0, 2, 2, 7], [6, 4, 3]  # the last has more rows than keys
    bt = np.array([[4, 1, 0], [2, 3, 0], [5, 0, 0]])
    kc, vc = rng.standard_normal((2, 6, page, hkv, D))
    q = rng.standard_normal((8, hq, D))
    out, lse, mag, smax = A.paged_attention(q, kc, vc, q_start, kv_len, bt, 0.7, causal, window)
    assert np.isnan(out[7]).all()
    for b in range(3):
        for t in range(q_start[b], q_start[b + 1]):
            p = kv_len[b] - q_start[b + 1] + t
            for h in range(hq):
                num, den, big = np.zeros(D), 0.0, 0.0
                for j in range(kv_len[b]):
                    if (causal and j > p) or (window and j <= p - window):
                        continue
                    k, v = (c[bt[b][j // page], j % page, h // 2] for c in (kc, vc))
                    e = math.exp(0.7 * float(q[t, h] @ k))
                    num, den = num + e * v, den + e
                    big = max(big, 0.7 * float(np.abs(q[t, h]) @ np.abs(k)))
                if den == 0:
                    assert np.array_equal(out[t, h], np.zeros(D)) and lse[t, h] == -math.inf
                else:
                    assert np.allclose(out[t, h], num / den) and math.isclose(lse[t, h], math.log(den))
                    assert math.isclose(smax[t, h], big) and (mag[t, h] + 1e-12 >= abs(out[t, h])).all()


def test_append_writes_only_its_slots():
    rng = np.random.default_rng(3)
    cache, rows = rng.standard_normal((4, 3, 2, 8)), rng.standard_normal((5, 2, 8))
    out = A.paged_append(cache, rows, [7, -1, 0, 12, 11])
    for slot, t in ((7, 0), (0, 2), (11, 4)):
        assert np.array_equal(out[slot // 3, slot % 3], rows[t])
    same = np.ones((4, 3), dtype=bool)
    same[7 // 3, 7 % 3] = same[0, 0] = same[11 // 3, 11 % 3] = False
    assert np.array_equal(out[same], cache[same])
