"""The comparison of attention over the 4-bit cache with the oracle tells wrong results from
right ones (no GPU needed): the mistakes are made in the oracle's results."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import test_gpu_attention
from helpers import to_f64
from oracle import attention as A
from oracle import mx4
from test_gpu_attention import ATTENTION, DT, MORE
from test_gpu_mx4_values import check_values

CASES = [(c, 0) for c in ATTENTION + MORE if sum(n * c[2] for n in c[0]) * max(c[1]) <= 1 << 18]
SIZES = [(c, e) for c, _ in CASES[1::8] for e in (-100, -60, 100)]


def _case(monkeypatch, args, e=0):
    """A case whose cache is what four bits stand for, garbage in the pages of no sequence."""
    q_lens, kv_lens, hq, hkv, D, page, dtype, causal, window, order = args
    monkeypatch.setattr(test_gpu_attention, "_randn", lambda rng, shape, dtype, scale=1.0: torch.from_numpy(
        (rng.standard_normal(shape) * scale).astype(np.float32)).to(DT[dtype]))
    c = test_gpu_attention._attention_case(q_lens, kv_lens, hq, hkv, D, page, dtype, order=order)
    used = np.zeros(c["n_pages"], dtype=bool)
    for b, n in enumerate(c["kv"]):
        used[c["bt"][b, :-(-int(n) // page)]] = True
    rng = np.random.default_rng(17)
    for n, up in (("k", 0), ("v", e)):
        codes, scales = mx4.encode(to_f64(c[n]) * 2.0 ** up)
        codes[~used] = rng.integers(0, 256, codes[~used].shape, dtype=np.uint8)
        scales[~used] = rng.integers(0, 256, scales[~used].shape, dtype=np.uint8)
        c[n] = torch.from_numpy(mx4.decode(codes, scales))
    out, lse, _, _ = A.paged_attention(to_f64(c["q"]), to_f64(c["k"]), to_f64(c["v"]), c["qs"], c["kv"],
                                       c["bt"], D ** -0.5, causal, window)
    return c, out, lse, (causal, window)


def _given(c, out, lse, mask):
    check_values(c, torch.from_numpy(out).to(DT[c["dtype"]]), torch.from_numpy(lse).float(), *mask)


def _refused(c, out, lse, mask):
    with pytest.raises(AssertionError):
        _given(c, out, lse, mask)


@pytest.mark.parametrize("args,e", CASES + SIZES)
def test_right_and_wrong_results(args, e, monkeypatch):
    """Values of 2^e."""
    c, out, lse, mask = _case(monkeypatch, args, e)
    _given(c, out, lse, mask)
    live = ~np.isneginf(lse)
    if not live.any():
        _refused(c, out - 3.0, lse, mask)
        return
    _refused(c, np.zeros_like(out), lse, mask)
    _refused(c, np.where(live[..., None], -3.0 * 2.0 ** e, 0.0), lse, mask)
    swapped = out.copy()
    swapped[..., [0, 1]] = out[..., [1, 0]]
    _refused(c, swapped, lse, mask)
    _refused(c, out * 1.05, lse, mask)
    if c["dims"][2] > 1 and (live & (lse != lse[:, ::-1])).any():   # another head's
        _refused(c, out[:, ::-1].copy(), lse, mask)
    _refused(c, out, np.where(live, lse + 0.1, lse), mask)
    row = tuple(np.argwhere(live)[0])
    for wrong in (math.nan, math.inf):
        one = out.copy()
        one[row][-1] = wrong
        _refused(c, one, lse, mask)
