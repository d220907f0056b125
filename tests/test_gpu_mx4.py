"""The 4-bit paged cache on the GPU against the float64 oracle.

What is stored is compared exactly: v is quantised without arithmetic, and k is computed in
64 bits and rounded to float32, which the oracle's float64 does too.  (They differ where
two 64-bit results straddle a float32 rounding border which in turn is a border of
codes: about 2^-53 / 2^-24 of one element in a few millions.)  What is read is compared
exactly: every stored value is a bfloat16 number.  Attention errs as over a cache of
values (test_gpu_attention.py), since decoding rounds nothing: the same tolerances, and one
absolute term.  A cache in four bits holds exact zeros, so that an element of a result may come
from keys of vanishing weight alone, and such weights are lost: float32 has no normal
numbers below 2^-126, and neither exp2 nor the matrix instructions need to keep the others.
Weights are relative to a running maximum that is at most the row's largest score, so that
their sum is at least 1 (2^-1 with its rounding): n of them lose at most n 2^-125 max |v|.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from helpers import to_f64
from oracle import attention as A
from oracle import mx4
from test_gpu_attention import (ATTENTION, DT, E, FEW_AND_MANY_ROWS, MORE, U, _attention_case,
                                _check_heads, _randn)

pytestmark = pytest.mark.gpu


def _mod():
    from activation_sparse_feed_amd import sffn
    return sffn


def _cache(rng, n_pages, page, hkv, D, order="head"):
    """A cache of arbitrary finite contents, in memory by head or by token."""
    sffn = _mod()
    shape = (n_pages, hkv, page) if order == "head" else (n_pages, page, hkv)
    t = []
    for _ in range(2):
        t.append(torch.from_numpy(rng.integers(0, 256, shape + (D // 2,), dtype=np.uint8)).cuda())
        t.append(torch.from_numpy(rng.integers(0, 253, shape + (mx4.blocks(D),), dtype=np.uint8)).cuda())
    if order == "head":
        t = [x.transpose(1, 2) for x in t]
    return sffn.Mx4Cache(n_pages, page, hkv, D, k_codes=t[0], k_scales=t[1], v_codes=t[2], v_scales=t[3])


def _held(cache, n):
    codes, scales = (getattr(cache, f"{n}_{x}").cpu().numpy() for x in ("codes", "scales"))
    return codes, scales


# ---------------------------------------------------------------- the append
@pytest.mark.parametrize("T,hq,hkv,D,rot,adjacent,norm,dtype,page,order", [
    (1, 8, 2, 128, 128, False, True, "bf16", 16, "head"),
    (70, 4, 4, 64, 64, False, True, "bf16", 1, "token"),
    (33, 0, 3, 80, 20, False, False, "f32", 24, "head"),     # no queries, rot / 2 = 10
    (2500, 5, 1, 128, 64, True, True, "bf16", 64, "head"),   # the many-token launch
    (9, 2, 1, 8, 8, False, True, "f32", 16, "token"),        # a block of eight
    (40, 3, 2, 16, 4, True, True, "f32", 5, "head"),
    (21, 6, 3, 96, 0, False, True, "bf16", 16, "head"),      # norm alone
    (50, 2, 2, 256, 36, False, True, "bf16", 16, "token"),   # rot / 2 = 18
    (50, 2, 5, 40, 40, True, False, "bf16", 16, "head"),     # rotation alone, a block of eight last
    (64, 2, 3, 112, 0, False, False, "f32", 16, "head"),     # neither
])
def test_append(T, hq, hkv, D, rot, adjacent, norm, dtype, page, order):
    sffn = _mod()
    rng = np.random.default_rng(T)
    n_pages = -(-T // page) + 4
    h = sffn.make_heads(T, hq, hkv, D, DT[dtype], rot, 4096 if rot else 0, norm, 1e-5, adjacent)
    qkv = _randn(rng, (T, hq + 2 * hkv, D), dtype)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    w = (1 + _randn(rng, (D,), "f32", 0.2)).to(DT[dtype]) if norm else None
    slots = rng.permutation(n_pages * page)[:T].astype(np.int32)
    slots[3::7] = -1
    if T > 20:
        slots[20] = n_pages * page      # past the cache: not stored
    pos = rng.integers(0, 4096, T).astype(np.int32)
    cache = _cache(rng, n_pages, page, hkv, D, order)
    before = {n: _held(cache, n) for n in "kv"}
    qo = torch.full((T, hq, D), math.nan, dtype=DT[dtype], device="cuda")
    tab = sffn.rotary_table(4096, rot) if rot else None
    sffn.paged_kv_append_mx4(h, q, k, v, w, w, tab, torch.from_numpy(pos).cuda(),
                             torch.from_numpy(slots).cuda(), qo, cache)
    wn, tn = None if w is None else to_f64(w), None if tab is None else to_f64(tab)
    case = (T, hq, hkv, D, rot, adjacent, norm, dtype, None)
    if hq:
        _check_heads(qo, to_f64(q), wn, tn, pos, case)
    eps = float(np.float32(1e-5))
    rows = {"k": A.norm_rope(to_f64(k), wn, tn, pos, rot, adjacent, norm, eps).astype(np.float32),
            "v": to_f64(v)}
    for n in "kv":
        want = [x.copy() for x in before[n]]
        for have, new in zip(want, mx4.encode(rows[n])):
            for t, slot in enumerate(slots):
                if 0 <= slot < n_pages * page:
                    have[slot // page, slot % page] = new[t]
        for a, b in zip(_held(cache, n), want):
            assert np.array_equal(a, b), (n, np.argwhere(a != b)[:4].tolist())


def test_quantising_limits():
    """Borders of the scale and of the codes, the largest and smallest numbers, NaN and
    infinities, as v of a float32 step; no row changes its neighbours."""
    sffn = _mod()
    rng = np.random.default_rng(1)
    T, D = 4096, 64
    e = rng.integers(-140, 128, (T, 1, 2, 1))
    mids = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7])
    x = np.ldexp(rng.choice(mids, (T, 1, 2, 32)) * rng.choice([-1.0, 1.0], (T, 1, 2, 32)), e)
    x = np.clip(x, -3.4028234e38, 3.4028234e38).astype(np.float32)
    near = rng.integers(0, 3, x.shape)
    x = np.where(near == 1, np.nextafter(x, np.float32(0)), np.where(near == 2, np.nextafter(
        x, np.sign(x) * np.float32(3.4028234e38)), x)).astype(np.float32).reshape(T, 1, D)
    x[5, 0, 3], x[6, 0, 40], x[7, 0, 63], x[8] = np.nan, np.inf, -np.inf, 0.0
    v = torch.from_numpy(x).cuda()
    cache = sffn.Mx4Cache(T // 16, 16, 1, D)
    h = sffn.make_heads(T, 0, 1, D, torch.float32)
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    sffn.paged_kv_append_mx4(h, None, v, v, None, None, None, None, slots, None, cache)
    codes, scales = mx4.encode(x)
    for n in "kv":
        c, s = _held(cache, n)
        assert np.array_equal(s.reshape(scales.shape), scales)
        assert np.array_equal(c.reshape(codes.shape), codes)


def test_what_is_stored_does_not_depend_on_the_call():
    """A token among many, among few, alone and in another head order gives the same bytes."""
    sffn = _mod()
    rng = np.random.default_rng(2)
    T, hkv, D = 2100, 4, 128
    q, k, v = (_randn(rng, (T, n, D), "bf16") for n in (8, hkv, hkv))
    w = (1 + _randn(rng, (D,), "f32", 0.2)).to(torch.bfloat16)
    tab = sffn.rotary_table(4096, D)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") + 7
    slots = torch.arange(T, dtype=torch.int32, device="cuda")

    def store(cache, lo, hi, n_q):
        h = sffn.make_heads(hi - lo, n_q, hkv, D, torch.bfloat16, D, 4096, True)
        qo = torch.empty((hi - lo, n_q, D), dtype=torch.bfloat16, device="cuda") if n_q else None
        sffn.paged_kv_append_mx4(h, q[lo:hi, :n_q] if n_q else None, k[lo:hi], v[lo:hi], w, w, tab,
                                 pos[lo:hi], slots[lo:hi], qo, cache)

    one, other = (sffn.Mx4Cache(T // 20, 20, hkv, D) for _ in range(2))
    store(one, 0, T, 8)
    store(other, 0, 1, 0)
    store(other, 1, 40, 3)
    store(other, 40, T, 5)
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert torch.equal(getattr(one, n), getattr(other, n))


def test_position_outside_the_table_is_nan():
    sffn = _mod()
    rng = np.random.default_rng(5)
    h = sffn.make_heads(4, 2, 1, 64, torch.bfloat16, 32, 10, True)
    q, k, v = (_randn(rng, (4, n, 64), "bf16") for n in (2, 1, 1))
    pos = torch.tensor([0, 10, -1, 9], dtype=torch.int32, device="cuda")
    slots = torch.arange(4, dtype=torch.int32, device="cuda")
    cache, qo = sffn.Mx4Cache(1, 4, 1, 64), torch.zeros_like(q)
    sffn.paged_kv_append_mx4(h, q, k, v, None, None, sffn.rotary_table(10, 32), pos, slots, qo, cache)
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    sffn.paged_kv_read_mx4(cache, slots, ko, vo)
    bad = torch.isnan(ko)
    assert bad[1:3, :, :32].all() and not bad[[0, 3]].any() and not bad[:, :, 32:].any()
    assert torch.isfinite(vo).all()


# ---------------------------------------------------------------- reading back
@pytest.mark.parametrize("T,hkv,D,dtype,page,order", [
    (1, 2, 128, "bf16", 16, "head"), (300, 3, 80, "f32", 24, "token"), (77, 1, 8, "bf16", 1, "head"),
    (40, 5, 256, "f32", 16, "head"), (1000, 2, 40, "bf16", 7, "head"), (64, 4, 64, "bf16", 16, "token"),
])
def test_read(T, hkv, D, dtype, page, order):
    """Every code under every scale that the types hold, into slices of larger tensors."""
    sffn = _mod()
    rng = np.random.default_rng(T)
    n_pages = -(-T // page) + 2
    cache = _cache(rng, n_pages, page, hkv, D, order)
    cache.v_scales[0] = 255
    cache.k_scales[1 % n_pages, :, :, -1] = 253
    slots = rng.integers(0, n_pages * page, T).astype(np.int32)     # some twice
    slots[2::5] = -1
    if T > 9:
        slots[8], slots[9] = n_pages * page, -2 ** 31
    out = torch.full((T, 2 * hkv + 1, D), 7.0, dtype=DT[dtype], device="cuda")
    sffn.paged_kv_read_mx4(cache, torch.from_numpy(slots).cuda(), out[:, :hkv], out[:, hkv:2 * hkv])
    got = out.float().cpu().numpy()
    keep = (slots >= 0) & (slots < n_pages * page)
    at = slots[keep] // page, slots[keep] % page
    for i, n in enumerate("kv"):
        codes, scales = _held(cache, n)
        want = mx4.decode(codes[at], scales[at]).astype(np.float32)
        assert np.array_equal(got[keep, i * hkv:(i + 1) * hkv], want, equal_nan=True)
    assert (got[~keep] == 7.0).all() and (got[:, 2 * hkv] == 7.0).all()
    # one of the two alone
    alone = torch.full((T, hkv, D), 7.0, dtype=DT[dtype], device="cuda")
    sffn.paged_kv_read_mx4(cache, torch.from_numpy(slots).cuda(), None, alone)
    assert torch.equal(torch.nan_to_num(alone, 5.0), torch.nan_to_num(out[:, hkv:2 * hkv], 5.0))


# ---------------------------------------------------------------- attention
def _quantised(c, order="head", garbage=True):
    """The case with its cache in four bits: c["k"], c["v"] are what that stands for.  What
    was not finite (behind a sequence's end, in pages of no sequence) is NaN, and of the pages of
    no sequence the bytes are arbitrary."""
    sffn = _mod()
    T, B, hq, hkv, D = c["dims"]
    rng = np.random.default_rng(17)
    used = np.zeros(c["n_pages"], dtype=bool)
    for b, n in enumerate(c["kv"]):
        used[c["bt"][b, :-(-int(n) // c["page"])]] = True
    t = []
    for n in "kv":
        codes, scales = mx4.encode(to_f64(c[n]))
        if garbage:
            codes[~used] = rng.integers(0, 256, codes[~used].shape, dtype=np.uint8)
            scales[~used] = rng.integers(0, 256, scales[~used].shape, dtype=np.uint8)
        c[n] = torch.from_numpy(mx4.decode(codes, scales))
        for x in (codes, scales):
            x = torch.from_numpy(x).cuda()
            t.append(x.transpose(1, 2).contiguous().transpose(1, 2) if order == "head" else x)
    c["cache"] = sffn.Mx4Cache(c["n_pages"], c["page"], hkv, D, k_codes=t[0], k_scales=t[1],
                               v_codes=t[2], v_scales=t[3])
    return c


def _case(*args, order="token", **kw):
    return _quantised(_attention_case(*args, **kw), "token" if order == "head" else "head")


def _run(c, causal=True, window=0, sm_scale=None, max_q=None, max_kv=None, lse=True):
    sffn = _mod()
    T, B, hq, hkv, D = c["dims"]
    b = sffn.make_paged_batch(T, B, hq, hkv, D, DT[c["dtype"]], c["page"], c["n_pages"],
                              c["bt"].shape[1], max_q or c["max_q"],
                              int(c["kv"].max()) if max_kv is None else max_kv, causal, window,
                              sm_scale)
    out = torch.full((T, hq, D), 7.0, dtype=DT[c["dtype"]], device="cuda")
    ls = torch.full((T, hq), 7.0, device="cuda") if lse else None
    ws = sffn.alloc_paged_mx4_workspace(b)
    ws.fill_(255)   # NaN everywhere: no initial contents are needed
    dev = [torch.from_numpy(c[n]).cuda() for n in ("qs", "kv", "bt")]
    sffn.paged_attn_mx4_fwd(b, c["q"], c["cache"], *dev, out, ws, lse=ls)
    torch.cuda.synchronize()
    return out, ls


def _check_attention(c, out, lse, causal=True, window=0, sm_scale=None):
    T, B, hq, hkv, D = c["dims"]
    s = D ** -0.5 if sm_scale is None else sm_scale
    v = to_f64(c["v"])
    want, want_l, mag, smax = A.paged_attention(to_f64(c["q"]), to_f64(c["k"]), v, c["qs"], c["kv"],
                                                c["bt"], s, causal, window)
    n = int(c["kv"].max())
    rel = 2 * ((D + 2) * smax + n + 64) * U + (2 * E if c["dtype"] == "bf16" else 0.0)
    own = E if c["dtype"] == "bf16" else U
    lost = n * 2.0 ** -125 * np.abs(v[np.isfinite(v)]).max(initial=0.0)
    rows = np.arange(T) < c["qs"][-1]
    got, got_l = to_f64(out), to_f64(lse)
    assert (got[~rows] == 7.0).all() and (got_l[~rows] == 7.0).all()
    empty = np.isneginf(want_l) & rows[:, None]
    assert (got[empty] == 0).all() and np.isneginf(got_l[empty]).all()
    live = rows[:, None] & ~empty
    err = np.abs(got - want)[live]
    tol = (own * np.abs(want) + (1 + own) * rel[..., None] * mag)[live] + lost
    assert (err <= tol).all(), (float(err.max()), float((err / tol).max()))
    errl = np.abs(got_l[live] - want_l[live])
    toll = (rel + 4 * U * np.abs(want_l))[live]
    assert (errl <= toll).all(), (float(errl.max()), float((errl / toll).max()))


@pytest.mark.parametrize("q_lens,kv_lens,hq,hkv,D,page,dtype,causal,window,order", ATTENTION + MORE)
def test_attention(q_lens, kv_lens, hq, hkv, D, page, dtype, causal, window, order):
    c = _case(q_lens, kv_lens, hq, hkv, D, page, dtype, order=order)
    out, lse = _run(c, causal, window)
    _check_attention(c, out, lse, causal, window)
    again, _ = _run(c, causal, window, lse=False)
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_lens,kv_lens,hq,hkv,D,page,window", FEW_AND_MANY_ROWS)
def test_few_and_many_rows(q_lens, kv_lens, hq, hkv, D, page, window, dtype):
    test_attention(q_lens, kv_lens, hq, hkv, D, page, dtype, True, window, "token")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_seqs,long", [(70, 0), (150, 5), (300, 0), (65, 65)])
def test_many_sequences(dtype, n_seqs, long):
    """More sequences than a wave has lanes, chunks among single tokens, empty ones."""
    rng = np.random.default_rng(n_seqs)
    q_lens = [1] * n_seqs
    for i in rng.permutation(n_seqs)[:long]:
        q_lens[i] = int(rng.integers(20, 60))
    kv_lens = [int(rng.integers(q, 300)) for q in q_lens]
    for i in (0, n_seqs // 2, n_seqs - 1):
        q_lens[i] = 0
    c = _case(q_lens, kv_lens, 8, 2, 64, 16, dtype, seed=n_seqs)
    out, lse = _run(c)
    _check_attention(c, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_padding_rows_are_left_alone(dtype):
    """Rows of q past the last sequence, as in a batch padded to a fixed size."""
    c = _case([3, 80, 30], [100, 90, 50], 4, 2, 64, 16, dtype, seed=21)
    c["qs"], c["kv"], c["bt"] = c["qs"][:3].copy(), c["kv"][:2].copy(), c["bt"][:2].copy()
    T, B, hq, hkv, D = c["dims"]
    c["dims"] = (T, 2, hq, hkv, D)
    out, lse = _run(c)
    _check_attention(c, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [16, 24])
def test_wrong_lengths_and_pages_stay_in_bounds(dtype, page):
    """Lengths beyond the stated bounds, rows out of range and pages that do not exist are
    cut to the bounds, and the sequences beside them come out right."""
    lens = ([1, 1, 40, 1, 90], [200, 64, 300, 90, 150])
    c = _case(*lens, 4, 2, 64, page, dtype, seed=22)
    good, good_l = _run(c)
    bad = dict(c, kv=c["kv"].copy(), qs=c["qs"].copy(), bt=c["bt"].copy())
    bad["kv"][1] = 1 << 30
    bad["kv"][3] = -5
    bad["bt"][2, :3] = [1 << 30, -7, c["n_pages"]]
    out, lse = _run(bad, max_kv=300)
    keep = [i for b in (0, 4) for i in range(c["qs"][b], c["qs"][b + 1])]
    assert torch.equal(out[keep], good[keep]) and torch.equal(lse[keep], good_l[keep])
    empty = int(c["qs"][3])
    assert (out[empty] == 0).all() and torch.isneginf(lse[empty]).all()
    bad = dict(c, qs=c["qs"].copy())
    bad["qs"][1:] = [-3, 1 << 30, 10, 43, 2000]
    _run(bad, max_q=90)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("max_q,max_kv", [(100, 512), (1000, 100 * 16)])
def test_bounds_of_the_lengths_are_upper_bounds(dtype, max_q, max_kv):
    c = _case([1, 40, 3], [500, 300, 512], 4, 2, 64, 16, dtype, seed=3)
    c["bt"] = np.concatenate([c["bt"], np.full((3, 100 - c["bt"].shape[1]), -5, np.int32)], 1)
    out, lse = _run(c, max_q=max_q, max_kv=max_kv)
    _check_attention(c, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_len", [1, 8, 150])
def test_large_scores(dtype, q_len):
    """Scores of several hundred: the running maximum keeps the sums finite."""
    c = _case([q_len], [700], 4, 2, 64, 16, dtype, seed=5, scale=40.0)
    out, lse = _run(c, sm_scale=0.3)
    _check_attention(c, out, lse, sm_scale=0.3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("sm_scale", [0.0, -0.2])
def test_zero_and_negative_scale(dtype, sm_scale):
    c = _case([1, 70, 9], [90, 130, 700], 4, 2, 80, 16, dtype, seed=6)
    out, lse = _run(c, sm_scale=sm_scale)
    _check_attention(c, out, lse, sm_scale=sm_scale)


NAN_BLOCKS = [
    # q_len, kv_len, D, page, window, keys: first tiles of a prompt, starts of windows, split
    # ranges, few rows; keys that all rows see
    (100, 100, 64, 16, 0, (0, 31, 40, 99)),
    (300, 300, 128, 16, 0, (5, 130)),
    (70, 70, 96, 24, 0, (0, 33)),
    (90, 90, 256, 16, 0, (33,)),
    (100, 700, 64, 16, 60, (541, 545, 600)),
    (90, 2800, 64, 8, 700, (2011, 2700)),
    (4, 60, 64, 16, 0, (0, 56, 58)),
    (4, 900, 128, 16, 100, (797, 798, 850)),
    (3, 9000, 128, 8, 0, (5000, 8997)),
    (2, 9000, 40, 16, 5000, (3999, 8998)),
    (7, 300, 256, 16, 0, (0, 296)),
    (1, 300, 80, 1, 0, (299,)),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_len,kv_len,D,page,window,keys", NAN_BLOCKS)
def test_nan_blocks_reach_the_rows_that_see_them(q_len, kv_len, D, page, window, keys, dtype):
    """A NaN block of a value is NaN in the results of the rows that see it and changes no
    other element or row; a NaN block of a key makes its rows NaN."""
    c = _case([q_len], [kv_len], 4, 2, D, page, dtype, seed=kv_len)
    clean, clean_l = _run(c, window=window)
    pos = torch.arange(kv_len - q_len, kv_len, device="cuda")
    for j in keys:
        seen = pos >= j
        if window:
            seen &= pos < j + window
        assert seen.any()
        at = int(c["bt"][0, j // page]), j % page
        for block, byte in ((0, 255), (mx4.blocks(D) - 1, 253)):
            kept = c["cache"].v_scales[at].clone()
            c["cache"].v_scales[at][:, block] = byte
            out, lse = _run(c, window=window)
            c["cache"].v_scales[at] = kept
            want = clean.clone()
            part = want[:, :, block * 32:block * 32 + 32]
            part[seen] = math.nan
            assert torch.equal(torch.isnan(out), torch.isnan(want)), (j, block)
            assert ((out == want) | torch.isnan(want)).all() and torch.equal(lse, clean_l)
        kept = c["cache"].k_scales[at].clone()
        c["cache"].k_scales[at][1, 0] = 255          # key head 1: query heads 2 and 3
        out, lse = _run(c, window=window)
        c["cache"].k_scales[at] = kept
        assert torch.isnan(out[seen][:, 2:]).all() and torch.isnan(lse[seen][:, 2:]).all()
        assert torch.equal(out[:, :2], clean[:, :2]) and torch.equal(out[~seen], clean[~seen])
        assert torch.equal(lse[:, :2], clean_l[:, :2]) and torch.equal(lse[~seen], clean_l[~seen])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_before_the_window_are_not_used(dtype):
    """Pages wholly before the window may be gone from the table, and rows before it in its
    first page may hold anything."""
    c = _case([3, 1, 50], [500, 400, 300], 4, 2, 64, 16, dtype, seed=8)
    out, lse = _run(c, window=100)
    _check_attention(c, out, lse, window=100)
    for b, (nq, n) in enumerate(((3, 500), (1, 400), (50, 300))):
        lo = n - nq - 100 + 1
        for j in range(lo):
            p = int(c["bt"][b, j // 16])
            c["cache"].k_scales[p, j % 16] = 255
            c["cache"].v_scales[p, j % 16] = 255 - j % 3
        c["bt"][b, :lo // 16] = -1
    again, again_l = _run(c, window=100)
    assert torch.equal(out, again) and torch.equal(lse, again_l)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("e", [-140, -60, 100])
def test_scales_near_the_ends_of_the_types(dtype, e):
    """Values of 2^e that a cache holds, with weights of a few keys: results keep their size."""
    c = _attention_case([1, 70], [300, 90], 4, 2, 64, 16, dtype, seed=9)
    c["v"] = torch.where(torch.isfinite(c["v"]), c["v"].double() * 2.0 ** e, math.nan)
    if e < -126:    # below 2^-125 the format's smallest scale rounds to multiples of 2^-125
        c["v"] = torch.where(torch.isfinite(c["v"]), c["v"] * 2.0 ** 16, math.nan)
    _quantised(c)
    out, lse = _run(c)
    _check_attention(c, out, lse)


def test_strides_of_every_order():
    """The same cache in other orders of page, token and head, K and V unlike each other, and as
    slices of larger buffers: the same bits."""
    sffn = _mod()
    c = _case([1, 5, 60], [300, 40, 200], 4, 2, 64, 16, "bf16", seed=13)
    want, want_l = _run(c)
    old = c["cache"]

    def laid(t, order, pad):
        big = torch.zeros([t.shape[o] + pad for o in order] + [t.shape[3] + 4 * pad], dtype=torch.uint8,
                          device="cuda")
        view = big[tuple(slice(0, t.shape[o]) for o in order) + (slice(0, t.shape[3]),)]
        view = view.permute(*[order.index(i) for i in range(3)], 3)
        view.copy_(t)
        return view

    names = ("k_codes", "k_scales", "v_codes", "v_scales")
    for orders in (((0, 1, 2),) * 4, ((2, 0, 1),) * 4, ((1, 2, 0), (0, 2, 1), (0, 2, 1), (2, 1, 0))):
        for pad in (0, 1):
            t = {n: laid(getattr(old, n), o, pad) for n, o in zip(names, orders)}
            c["cache"] = sffn.Mx4Cache(old.n_pages, 16, 2, 64, **t)
            out, lse = _run(c)
            assert torch.equal(out, want) and torch.equal(lse, want_l)


def test_on_a_side_stream_and_in_a_graph():
    """A whole step, append and attention, captured once and replayed with changing inputs
    and eager work between; the read-back beside it."""
    sffn = _mod()
    rng = np.random.default_rng(11)
    B, hq, hkv, D, page = 3, 8, 2, 128, 16
    c = _case([1] * B, [900, 40, 300], hq, hkv, D, page, "bf16", seed=11)
    att = sffn.PagedAttention(B, B, hq, hkv, D, torch.bfloat16, page, c["n_pages"], c["bt"].shape[1], 1,
                              900, rot_dim=D, max_pos=1000, norm=True, mx4=c["cache"])
    qkv = _randn(rng, (B, hq + 2 * hkv, D), "bf16")
    tab, bt = sffn.rotary_table(1000, D), torch.from_numpy(c["bt"]).cuda()
    qs, kv = torch.from_numpy(c["qs"]).cuda(), torch.from_numpy(c["kv"]).cuda()
    slots, pos = torch.empty(B, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
    ko, vo = (torch.empty((B, hkv, D), device="cuda") for _ in range(2))

    def step():
        att.forward(qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], pos, slots, qs, kv, bt, tab)
        sffn.paged_kv_read_mx4(c["cache"], slots, ko, vo)

    def check():
        torch.cuda.synchronize()
        codes, scales = mx4.encode(to_f64(qkv[:, hq + hkv:]))
        assert np.array_equal(vo.cpu().numpy(), mx4.decode(codes, scales).astype(np.float32))
        for n in "kv":
            c[n] = torch.from_numpy(mx4.decode(*_held(c["cache"], n)))
        _check_attention(dict(c, q=att.q_out), att.out, att.lse)

    def lengths(lens):
        c["kv"] = np.array(lens, dtype=np.int32)
        kv.copy_(torch.from_numpy(c["kv"]))
        pos.copy_(kv - 1)
        slots.copy_(sffn.paged_slots(bt, torch.arange(B, device="cuda"), pos, page))

    lengths([900, 40, 300])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for lens in ([900, 40, 300], [1, 33, 299], [555, 2, 150], [900, 40, 300]):
        lengths(lens)
        qkv.normal_()
        att.out.zero_()
        g.replay()
        check()


def test_cache_beyond_four_gib():
    """Byte offsets past 32 bits, in the append, the read-back and the attention."""
    sffn = _mod()
    page, hkv, D = 64, 8, 256
    n_pages = (5 << 30) // (page * hkv * D // 2)
    cache = sffn.Mx4Cache(n_pages, page, hkv, D)
    rng = np.random.default_rng(12)
    T = 100
    qkv = _randn(rng, (T, 3 * hkv, D), "bf16")
    q, k, v = qkv[:, :hkv], qkv[:, hkv:2 * hkv], qkv[:, 2 * hkv:]
    pages = np.array([n_pages - 1, n_pages // 2 + 3], dtype=np.int32)
    slots = torch.from_numpy((pages[np.arange(T) // page] * page + np.arange(T) % page).astype(np.int32)).cuda()
    h = sffn.make_heads(T, hkv, hkv, D, torch.bfloat16)
    qo = torch.empty((T, hkv, D), dtype=torch.bfloat16, device="cuda")
    sffn.paged_kv_append_mx4(h, q, k, v, None, None, None, None, slots, qo, cache)
    ko, vo = torch.empty_like(qo), torch.empty_like(qo)
    sffn.paged_kv_read_mx4(cache, slots, ko, vo)
    for x, y in ((k, ko), (v, vo)):
        assert np.array_equal(to_f64(y), mx4.decode(*mx4.encode(to_f64(x))))
    small = sffn.Mx4Cache(2, page, hkv, D)
    at = torch.from_numpy(pages).cuda().long()
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        getattr(small, n).copy_(getattr(cache, n)[at])
    c = {"q": q, "cache": small, "bt": np.array([[0, 1]], np.int32), "kv": np.array([T], np.int32),
         "qs": np.array([0, T], np.int32), "page": page, "n_pages": 2, "dims": (T, 1, hkv, hkv, D),
         "dtype": "bf16", "max_q": T}
    o1, l1 = _run(c)
    o2, l2 = _run(dict(c, cache=cache, bt=pages[None, :].copy(), n_pages=n_pages))
    assert torch.equal(o1, o2) and torch.equal(l1, l2)
    one = dict(c, q=q[:1], dims=(1, 1, hkv, hkv, D), qs=np.array([0, 1], np.int32), max_q=1)
    o1, l1 = _run(one)
    o2, l2 = _run(dict(one, cache=cache, bt=pages[None, :].copy(), n_pages=n_pages))
    assert torch.equal(o1, o2) and torch.equal(l1, l2)


# ------------------------------------------------- float32 first, 64 bits where it matters
@pytest.mark.parametrize("dtype,adjacent,weights,eps", [
    ("bf16", False, True, 1e-6), ("f32", False, True, 1e-6), ("f32", True, False, 1e-6), ("f32", False, False, 0.0)])
def test_many_codes_are_those_of_64_bits(dtype, adjacent, weights, eps):
    """Three million elements: tens of them lie closer to a border between two codes than
    float32 arithmetic can tell."""
    sffn = _mod()
    rng = np.random.default_rng(77)
    T, hkv, D = 3000, 8, 128
    k = _randn(rng, (T, hkv, D), dtype)
    k *= torch.exp2(torch.from_numpy(rng.integers(-8, 8, (T, hkv, 1))).cuda()).to(k.dtype)
    w = (1 + _randn(rng, (D,), "f32", 0.3)).to(DT[dtype]) if weights else None
    tab = sffn.rotary_table(5000, D)
    pos = rng.integers(0, 5000, T).astype(np.int32)
    cache = sffn.Mx4Cache(-(-T // 16), 16, hkv, D)
    h = sffn.make_heads(T, 0, hkv, D, DT[dtype], D, 5000, True, eps, adjacent)
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    sffn.paged_kv_append_mx4(h, None, k, k, None, w, tab, torch.from_numpy(pos).cuda(), slots, None, cache)
    rows = A.norm_rope(to_f64(k), None if w is None else to_f64(w), to_f64(tab), pos, D, adjacent, True,
                       float(np.float32(eps)))
    codes, scales = mx4.encode(rows.astype(np.float32))
    c, s = _held(cache, "k")
    assert np.array_equal(s.reshape(-1, hkv, 4)[:T], scales)
    assert np.array_equal(c.reshape(-1, hkv, D // 2)[:T], codes)


@pytest.mark.parametrize("size", [1e-40, 1e-30, 1e-20, 1e-10, 1e10, 1e18, 1e30])
@pytest.mark.parametrize("weight", [1e-30, 1.0, 1e20])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_sizes_at_which_float32_squares_or_products_fail(size, weight, eps):
    """Rows whose squares overflow or vanish in float32, weights that take products to its
    ends: the codes are those of 64 bits."""
    sffn = _mod()
    rng = np.random.default_rng(78)
    T, hkv, D, rot = 40, 3, 80, 40
    x = (rng.standard_normal((T, hkv, D)) * size).astype(np.float32)
    x[3, 1], x[4, 0, 5:9], x[5, 2] = 0.0, 0.0, rng.standard_normal(D).astype(np.float32)
    x[6, 0, :32] *= np.float32(1e-8)
    k = torch.from_numpy(x).cuda()
    w = torch.from_numpy(((1 + 0.3 * rng.standard_normal(D)) * weight).astype(np.float32)).cuda()
    tab = sffn.rotary_table(100, rot)
    pos = rng.integers(0, 100, T).astype(np.int32)
    cache = sffn.Mx4Cache(3, 16, hkv, D)
    h = sffn.make_heads(T, 0, hkv, D, torch.float32, rot, 100, True, eps)
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    sffn.paged_kv_append_mx4(h, None, k, k, None, w, tab, torch.from_numpy(pos).cuda(), slots, None, cache)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        rows = A.norm_rope(x.astype(np.float64), to_f64(w), to_f64(tab), pos, rot, False, True,
                           float(np.float32(eps))).astype(np.float32)
    codes, scales = mx4.encode(rows)
    c, s = _held(cache, "k")
    assert np.array_equal(s.reshape(-1, hkv, 3)[:T], scales)
    assert np.array_equal(c.reshape(-1, hkv, D // 2)[:T], codes)
