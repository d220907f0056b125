"""Values of attention over the 4-bit cache against the float64 oracle, within bounds that are
each row's own.

The bounds are those of attention over a cache of values (test_gpu_attention.py) and one
absolute term, for what float32 loses below its normal numbers: weights relative to the running
maximum below 2^-126, and products with them.  The maximum is at most the row's largest score,
so that the weights' sum is at least 1 (2^-1 with its rounding), and n keys lose at most
n 2^-125 (1 + |v|) of an element, with the largest |v| of that element among the keys that the
row sees.  (With the largest of the whole cache, whose unused pages hold anything, the term
would pass for every result.)  Beside the largest error that there can be, which over thousands of
keys is as large as the result, its norm is compared as for a cache of values: single
roundings are as often up as down.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import test_gpu_mx4 as M
from helpers import to_f64
from oracle import attention as A
from test_gpu_attention import ATTENTION, E, FEW_AND_MANY_ROWS, MORE, U, _attention_case

pytestmark = pytest.mark.gpu

TYPICAL = {"bf16": 5e-3, "f32": 1e-5}    # of the results' norm


def largest_values(c, causal=True, window=0):
    """The largest |v| of every element among the keys that a row sees, [T, hq, D]."""
    T, B, hq, hkv, D = c["dims"]
    v, res = np.abs(to_f64(c["v"])), np.zeros((T, hq, D))
    for b in range(B):
        r0, r1, n = int(c["qs"][b]), int(c["qs"][b + 1]), int(c["kv"][b])
        j = np.arange(n)
        x = v[c["bt"][b][j // c["page"]], j % c["page"]] if n else np.zeros((0, hkv, D))
        for t in range(r0, r1):
            pos = n - r1 + t
            hi = max(pos + 1, 0) if causal else n
            lo = min(max(pos - window + 1, 0), hi) if window > 0 else 0
            if hi > lo:
                res[t] = np.repeat(x[lo:hi].max(0), hq // hkv, 0)
    return res


def check_values(c, out, lse, causal=True, window=0, sm_scale=None, lost=None):
    T, B, hq, hkv, D = c["dims"]
    s = D ** -0.5 if sm_scale is None else sm_scale
    want, want_l, mag, smax = A.paged_attention(to_f64(c["q"]), to_f64(c["k"]), to_f64(c["v"]), c["qs"],
                                                c["kv"], c["bt"], s, causal, window)
    n = int(c["kv"].max())
    rel = 2 * ((D + 2) * smax + n + 64) * U + (2 * E if c["dtype"] == "bf16" else 0.0)
    own = E if c["dtype"] == "bf16" else U
    if lost is None:
        lost = n * 2.0 ** -125 * (1.0 + largest_values(c, causal, window))
    lost = np.broadcast_to(lost, want.shape)
    rows = np.arange(T) < c["qs"][-1]
    got, got_l = to_f64(out), to_f64(lse)
    assert (got[~rows] == 7.0).all() and (got_l[~rows] == 7.0).all()
    empty = np.isneginf(want_l) & rows[:, None]
    assert (got[empty] == 0).all() and np.isneginf(got_l[empty]).all()
    live = rows[:, None] & ~empty
    err = np.abs(got - want)[live]
    tol = (own * np.abs(want) + (1 + own) * rel[..., None] * mag + lost)[live]
    assert (err <= tol).all(), (float(err.max()), float((err / tol).max()))
    if live.any():
        norm, bound = np.linalg.norm(err), TYPICAL[c["dtype"]] * np.linalg.norm(want[live])
        assert norm <= bound + np.linalg.norm(lost[live]), (norm, bound)
    errl = np.abs(got_l[live] - want_l[live])
    toll = (rel + 4 * U * np.abs(want_l))[live]
    assert (errl <= toll).all(), (float(errl.max()), float((errl / toll).max()))


@pytest.fixture(autouse=True)
def own_bounds(monkeypatch):
    monkeypatch.setattr(M, "_check_attention", check_values)


@pytest.mark.parametrize("q_lens,kv_lens,hq,hkv,D,page,dtype,causal,window,order", ATTENTION + MORE)
def test_attention(q_lens, kv_lens, hq, hkv, D, page, dtype, causal, window, order):
    M.test_attention(q_lens, kv_lens, hq, hkv, D, page, dtype, causal, window, order)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_lens,kv_lens,hq,hkv,D,page,window", FEW_AND_MANY_ROWS)
def test_few_and_many_rows(q_lens, kv_lens, hq, hkv, D, page, window, dtype):
    M.test_few_and_many_rows(q_lens, kv_lens, hq, hkv, D, page, window, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [16, 48, 88, 96, 160, 192, 224, 256])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 3], [700, 65]), ([90, 1], [300, 40])])
def test_widths(q_lens, kv_lens, D, dtype):
    M.test_attention(q_lens, kv_lens, 6, 2, D, 16 if D % 32 else 24, dtype, True, 0, "token")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_seqs,long", [(70, 0), (150, 5), (300, 0), (65, 65)])
def test_many_sequences(dtype, n_seqs, long):
    M.test_many_sequences(dtype, n_seqs, long)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_padding_rows_are_left_alone(dtype):
    M.test_padding_rows_are_left_alone(dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("max_q,max_kv", [(100, 512), (1000, 100 * 16)])
def test_bounds_of_the_lengths_are_upper_bounds(dtype, max_q, max_kv):
    M.test_bounds_of_the_lengths_are_upper_bounds(dtype, max_q, max_kv)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_len", [1, 8, 150])
def test_large_scores(dtype, q_len):
    M.test_large_scores(dtype, q_len)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("sm_scale", [0.0, -0.2])
def test_zero_and_negative_scale(dtype, sm_scale):
    M.test_zero_and_negative_scale(dtype, sm_scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_before_the_window_are_not_used(dtype):
    M.test_rows_before_the_window_are_not_used(dtype)


def test_on_a_side_stream_and_in_a_graph():
    M.test_on_a_side_stream_and_in_a_graph()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 70], [300, 90]), ([3, 1], [2500, 40])])
@pytest.mark.parametrize("e", [-100, -60, -20, 20, 60, 100])
def test_values_of_all_sizes(e, q_lens, kv_lens, dtype):
    """Values of 2^e: every result has its size.  (At -100 the absolute term is up to 2^-14 of
    it, from -60 on nothing.)"""
    c = _attention_case(q_lens, kv_lens, 4, 2, 64, 16, dtype, seed=9)
    c["v"] = torch.where(torch.isfinite(c["v"]), c["v"].double() * 2.0 ** e, math.nan)
    M._quantised(c)
    out, lse = M._run(c)
    check_values(c, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 70], [300, 90]), ([3, 1], [2500, 40])])
def test_smallest_values(q_lens, kv_lens, dtype):
    """Values of 2^-124, near the smallest that a cache holds: the matrix instructions keep
    subnormal products to multiples of 2^-149, with a sum of weights of at least 2^-1 n 2^-148 of a
    result, which is rounded to multiples of 2^-133 (bf16) or 2^-149."""
    c = _attention_case(q_lens, kv_lens, 4, 2, 64, 16, dtype, seed=9)
    c["v"] = torch.where(torch.isfinite(c["v"]), c["v"].double() * 2.0 ** -124, math.nan)
    M._quantised(c)
    out, lse = M._run(c)
    check_values(c, out, lse, lost=max(kv_lens) * 2.0 ** -148 + (2.0 ** -134 if dtype == "bf16" else 2.0 ** -150))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sequences_of_unlike_sizes(dtype):
    """Large values of one sequence and key head say nothing about the others' results."""
    c = _attention_case([1, 40, 2], [300, 90, 700], 4, 2, 64, 16, dtype, seed=10)
    v = c["v"].double()
    for b, e in enumerate((-60, 100, 0)):
        for p in c["bt"][b, :-(-int(c["kv"][b]) // 16)]:
            v[int(p)] *= 2.0 ** e
            v[int(p), :, 1] *= 2.0 ** -16
    c["v"] = torch.where(torch.isfinite(v), v, math.nan)
    M._quantised(c)
    out, lse = M._run(c)
    check_values(c, out, lse)
