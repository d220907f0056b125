"""The 4-bit paged cache on the GPU against the float64 oracle.

What is stored is compared exactly: v is quantised without arithmetic, and k is computed in
64 bits and rounded to float32, which the oracle's float64 does too.  (They differ where
two 64-bit results straddle a float32 rounding border which in turn is a border of
codes: about 2^-53 / 2^-24 of one element in a few millions.)  What is read is compared
exactly: every stored value is a bfloat16 number.  Attention errs as over a cache of
values (test_gpu_attention.py), since decoding rounds nothing: the same tolerances.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from helpers import to_f64
from oracle import attention as A
from oracle import mx4
from test_gpu_attention import (ATTENTION, DT, FEW_AND_MANY_ROWS, MORE, _attention_case,
                                _check_attention, _check_heads, _randn)

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
