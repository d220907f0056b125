"""Infinities, NaN and extreme limits in paged_attn_fwd: results that follow from the
definition without rounding, so they are compared exactly."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from test_gpu_attention import _attention_case, _check_attention, _run

pytestmark = pytest.mark.gpu


INFINITE = [
    # q_len, kv_len, D, page, window, keys
    # the first tiles of a prompt, which the first rows see in part
    (100, 100, 64, 16, 0, (0, 1, 31, 40, 63, 64)),
    (300, 300, 128, 16, 0, (0, 5, 130)),
    (70, 70, 96, 24, 0, (0, 33)),
    (90, 90, 256, 16, 0, (0, 33)),
    # the start of a window
    (100, 700, 64, 16, 60, (541, 545, 600)),
    # split ranges, from the start and from inside a window
    (100, 3000, 128, 16, 0, (0, 2900, 2950)),
    (90, 2800, 64, 8, 700, (2011, 2040, 2700)),
    # few rows
    (4, 60, 64, 16, 0, (0, 56, 58)),
    (4, 900, 128, 16, 100, (797, 798, 850)),
    (3, 9000, 128, 8, 0, (0, 5000, 8997)),
    (2, 9000, 64, 16, 5000, (3999, 4500, 8998)),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("q_len,kv_len,D,page,window,keys", INFINITE)
def test_infinite_values_reach_the_rows_that_see_them(q_len, kv_len, D, page, window, keys, bad, dtype):
    """An infinite element of a value is the result's for every row that sees it (a
    positive weight times infinity), and everything else is as without it."""
    c = _attention_case([q_len], [kv_len], 4, 2, D, page, dtype, seed=kv_len)
    clean, clean_l = _run(c, window=window)
    pos = torch.arange(kv_len - q_len, kv_len, device="cuda")
    for j in keys:
        at = c["v"][int(c["bt"][0, j // page]), j % page]
        kept = at.clone()
        at[:, 3::5] = bad
        out, lse = _run(c, window=window)
        at.copy_(kept)
        seen = pos >= j
        if window:
            seen &= pos < j + window
        assert seen.any()
        want = clean.clone()
        part = want[:, :, 3::5]
        part[seen] = bad
        assert torch.equal(torch.isnan(out), torch.isnan(want))
        same = (out == want) | torch.isnan(want)
        assert same.all(), (j, (~same).nonzero()[:4].tolist())
        assert torch.equal(lse, clean_l)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_len,kv_len", [(1, 300), (1, 9001), (100, 200), (100, 3000)])
def test_nan_of_vanishing_weight_is_not_lost(q_len, kv_len, dtype):
    """The first half of the keys has scores of -800, whose weights are 0 in float32; a
    NaN among their values is the result's all the same, whether or not these keys are
    a split of their own."""
    c = _attention_case([q_len], [kv_len], 4, 2, 64, 16, dtype, seed=kv_len)
    c["q"][:] = 1.0
    for j in range(kv_len // 2):
        c["k"][int(c["bt"][0, j // 16]), j % 16] = -100.0   # scores of -100 * 64 / 8
    clean, clean_l = _run(c)
    c["v"][int(c["bt"][0, 0]), 10, :, 3::5] = math.nan
    out, lse = _run(c)
    bad = torch.zeros(64, dtype=torch.bool, device="cuda")
    bad[3::5] = True
    assert torch.isnan(out[:, :, bad]).all()
    assert torch.equal(out[:, :, ~bad], clean[:, :, ~bad]) and torch.equal(lse, clean_l)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 40, 1 << 30, 1500])
@pytest.mark.parametrize("q_lens,kv_lens", [([5, 1, 40], [2, 900, 33]), ([150, 3], [20, 1500])])
def test_windows_that_hide_nothing(q_lens, kv_lens, window, causal, dtype):
    """A window of at least every sequence's length is none, up to the largest number, also
    where a sequence has more rows than keys (its first positions are negative)."""
    c = _attention_case(q_lens, kv_lens, 4, 2, 64, 16, dtype, seed=31)
    out, lse = _run(c, causal, window)
    _check_attention(c, out, lse, causal, window)
    free, free_l = _run(c, causal, 0)
    assert torch.equal(out, free) and torch.equal(lse, free_l)


@pytest.mark.parametrize("D", [96, 192])
@pytest.mark.parametrize("q_lens,kv_lens,window", [([2000], [2000], 200), ([1, 3, 40, 2], [900, 300, 500, 2000], 0)])
def test_widths_between_the_lds_rows(D, q_lens, kv_lens, window):
    """Rows of 96 and 192 elements leave a part of their LDS rows unused."""
    c = _attention_case(q_lens, kv_lens, 4, 2, D, 16, "bf16", seed=D)
    out, lse = _run(c, window=window)
    _check_attention(c, out, lse, window=window)


def test_time_does_not_depend_on_what_lds_held():
    """A prompt of width 96 in a window after a call that leaves infinities everywhere in LDS
    takes as long as after one that leaves finite numbers: the unused part of an LDS row is not
    searched for them.  Medians of 15, and a factor of two for noise (it was five)."""
    from activation_sparse_feed_amd import sffn

    def call(D, n, window, value=None):
        c = _attention_case([n], [n], 16, 4, D, 16, "bf16", seed=D)
        if value is not None:
            c["k"].fill_(value)
            c["v"].fill_(value)
        b = sffn.make_paged_batch(n, 1, 16, 4, D, torch.bfloat16, 16, c["n_pages"], c["bt"].shape[1],
                                  n, n, window=window)
        dev = [torch.from_numpy(c[x]).cuda() for x in ("qs", "kv", "bt")]
        out, ws = torch.empty((n, 16, D), dtype=torch.bfloat16, device="cuda"), sffn.alloc_paged_workspace(b)
        return lambda: sffn.paged_attn_fwd(b, c["q"], c["k"], c["v"], *dev, out, ws)

    timed = call(96, 4096, 300)
    medians = []
    for value in (1.0, math.inf):
        before, times = call(256, 1024, 0, value), []
        for _ in range(15):
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            before()
            start.record()
            timed()
            end.record()
            torch.cuda.synchronize()
            times.append(start.elapsed_time(end))
        medians.append(sorted(times)[7])
    assert medians[1] < 2 * medians[0], medians


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_sequences_under_the_limit_of_a_model(dtype):
    """1100 sequences, most of them short, with max_kv far above them: the partial results are
    limited, so that the few long ones are split less often than alone."""
    rng = np.random.default_rng(40)
    q_lens = [int(n) for n in rng.integers(1, 5, 1100)]
    kv_lens = [int(n) for n in rng.integers(4, 60, 1100)]
    for i, n in ((0, 20000), (500, 9500), (1099, 12001)):
        kv_lens[i] = n
    c = _attention_case(q_lens, kv_lens, 8, 1, 128, 16, dtype, seed=41)
    c["bt"] = np.concatenate([c["bt"], np.full((1100, 8192 - c["bt"].shape[1]), -1, np.int32)], 1)
    out, lse = _run(c, max_kv=131072)
    _check_attention(c, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 3], [90, 5000]), ([100], [130])])
@pytest.mark.parametrize("size,sm_scale", [(1e14, 1e-29), (1e14, -3e-29), (1e18, 0.0), (1e17, 1e-35)])
def test_very_small_scales(q_lens, kv_lens, size, sm_scale, dtype):
    """Scores count after their scale, however small it is: products of 1e29 times 1e-29, and
    a scale of 0, which makes every key's weight the same, with products of 1e36."""
    c = _attention_case(q_lens, kv_lens, 4, 2, 64, 16, dtype, seed=50, scale=size)
    finite = torch.isfinite(c["k"])
    c["k"] = torch.where(finite, c["k"] * size, c["k"])
    out, lse = _run(c, sm_scale=sm_scale)
    _check_attention(c, out, lse, sm_scale=sm_scale)
