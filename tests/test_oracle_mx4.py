"""The oracle of the 4-bit cache format against the definition's consequences (CPU)."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import mx4


def test_every_value_stands_for_itself():
    """Values that a block can hold come back unchanged, whatever its largest one."""
    for top in (4.0, 6.0):
        for e in (-124, -3, 0, 60, 125):
            x = np.zeros((1, 32))
            x[0, :15] = np.concatenate([mx4.MAGNITUDES, -mx4.MAGNITUDES[1:]])
            x[np.abs(x) > top] = 0
            x *= 2.0 ** e
            codes, scales = mx4.encode(x)
            assert scales[0, 0] == e + 127
            assert np.array_equal(mx4.decode(codes, scales), x)


def test_codes_by_hand():
    x = np.zeros((1, 32))
    x[0, :10] = [6, -0.5, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.1]
    codes, scales = mx4.encode(x)
    assert scales[0, 0] == 127
    # ties to the even code: .25 -> 0, .75 -> 1 (2), 1.25 -> 1 (2), 1.75 -> 2 (4), 2.5 -> 2 (4),
    # 3.5 -> 4 (6), 5 -> 4 (6); -.1 -> -0 (8)
    assert codes[0, :5].tolist() == [7 | 9 << 4, 0 | 2 << 4, 2 | 4 << 4, 4 | 6 << 4, 6 | 8 << 4]


@pytest.mark.parametrize("dim", [8, 32, 40, 80, 128, 256])
def test_error_is_half_a_step(dim):
    rng = np.random.default_rng(dim)
    x = rng.standard_normal((50, 3, dim)) * np.exp2(rng.integers(-20, 20, (50, 1, 1)))
    codes, scales = mx4.encode(x)
    assert codes.shape == (50, 3, dim // 2) and scales.shape == (50, 3, -(-dim // 32))
    y = mx4.decode(codes, scales)
    e = np.repeat(scales.astype(np.float64) - 127, 32, -1)[..., :dim]
    m = np.abs(x) / np.exp2(e)
    assert (m < 7).all()
    step = np.where(m < 2, 0.5, np.where(m < 4, 1.0, 2.0))
    assert (np.abs(x - y) <= step / 2 * np.exp2(e)).all()
    # the exponent is the smallest that holds the largest element
    top = np.abs(x).reshape(50, 3, -1)
    for b in range(scales.shape[-1]):
        t = top[..., b * 32:(b + 1) * 32].max(-1)
        assert (t >= 3.5 * np.exp2(scales[..., b] - 127.0)).all()


def test_limits():
    x = np.zeros((6, 8))
    x[0, 0] = np.nan
    x[1, 3] = -np.inf
    x[2, :2] = [3e38, -1e38]          # over 7 * 2^125: saturated
    x[3, :2] = [2.0 ** -126, -2.0 ** -124]
    x[4, 0] = 1e-45
    codes, scales = mx4.encode(x)
    assert scales[:, 0].tolist() == [255, 255, 252, 3, 3, 3]
    y = mx4.decode(codes, scales)
    assert np.isnan(y[:2]).all()
    assert y[2, :2].tolist() == [6 * 2.0 ** 125, -2 * 2.0 ** 125]
    assert y[3, :2].tolist() == [0.0, -2.0 ** -124]   # a quarter of a step: a tie, to 0
    assert (y[4:] == 0).all()
    assert np.isnan(mx4.decode(codes[5], np.array([253], np.uint8))).all()
