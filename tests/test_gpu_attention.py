"""The attention side of the block on the GPU against the float64 oracle.

Tolerances, u = 2^-24 (float32) and e = 2^-8 (half an ulp of bf16, relative):

* an output in bf16 is rounded once: e |y|; in float32 the same with u.
* norm and rotation: every element is a sum of two products of a normalised
  element; the mean square of D values errs by at most D u relative (half of
  that in its root), the rest by a handful of u: (D + 16) u of |n_a| + |n_b|.
* attention: a score errs by (D + 2) u of its sum of |q k| (`smax`, scaled), and
  a weight by that and by some u for the exponential; a sum over n keys by n u;
  bf16 weights are rounded, e each.  Applied to the weighted mean of |v|
  (`mag`), numerator and denominator: 2 ((D + 2) smax + n + 64) u + 2 e.
* lse: the same without the bf16 rounding of the weights (its sum may be of
  rounded weights: e), plus u of its own size.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from helpers import to_f64
from oracle import attention as A

pytestmark = pytest.mark.gpu

U, E = 2.0 ** -24, 2.0 ** -8
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _randn(rng, shape, dtype, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).cuda().to(DT[dtype])


def _mod():
    from activation_sparse_feed_amd import sffn
    return sffn


# ---------------------------------------------------------------- norm, rotation
def _magnitude(x, w, rot, adjacent, norm, eps):
    """|n_a| + |n_b| of every element's pair (|n| of an unrotated one)."""
    n = x
    if norm:
        n = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1.0 if w is None else w)
    m = np.abs(n)
    if rot:
        a, b = A.pair_indices(rot, adjacent)
        m[..., a] = m[..., b] = m[..., a] + m[..., b]
    return m


HEADS = [
    # T, hq, hkv, D, rot, adjacent, norm, dtype, weights
    (1, 32, 8, 128, 128, False, True, "bf16", True),
    (37, 16, 4, 128, 64, False, True, "bf16", True),
    (5, 3, 1, 80, 20, False, True, "bf16", True),     # rot / 2 = 10: chunks of two elements
    (9, 5, 5, 80, 40, False, True, "bf16", False),    # rot / 2 = 20: chunks of four
    (300, 7, 7, 64, 64, True, True, "bf16", True),
    (33, 4, 2, 72, 44, True, True, "f32", True),
    (64, 2, 1, 256, 256, False, True, "f32", True),
    (11, 1, 1, 256, 36, False, True, "f32", False),   # rot / 2 = 18: chunks of two elements
    (21, 6, 2, 8, 8, False, True, "f32", True),
    (21, 6, 2, 8, 4, False, True, "bf16", True),
    (21, 6, 2, 96, 0, False, True, "bf16", True),     # norm alone
    (50, 8, 2, 128, 128, False, False, "bf16", False),  # rotation alone
    (50, 8, 2, 112, 96, True, False, "f32", False),
    (2100, 9, 3, 64, 64, False, True, "bf16", True),  # the many-token launch
    (13, 8, 0, 64, 64, False, True, "bf16", True),    # q only
    (13, 0, 8, 64, 64, False, True, "bf16", True),    # k only
]


def _heads_case(case, seed=0):
    T, hq, hkv, D, rot, adjacent, norm, dtype, weights = case
    rng = np.random.default_rng(seed)
    sffn = _mod()
    max_pos = 500
    c = {"h": sffn.make_heads(T, hq, hkv, D, DT[dtype], rot, max_pos if rot else 0, norm, 1e-5, adjacent)}
    # q and k are slices of one projection, with a value head between them
    qkv = _randn(rng, (T, hq + hkv + 2, D), dtype)
    c["q"], c["k"] = qkv[:, :hq], qkv[:, hq + 1:hq + 1 + hkv]
    c["wq"] = (1 + _randn(rng, (D,), "f32", 0.3)).to(DT[dtype]) if weights else None
    c["wk"] = (1 + _randn(rng, (D,), "f32", 0.3)).to(DT[dtype]) if weights else None
    c["table"] = sffn.rotary_table(max_pos, rot) if rot else None
    c["pos"] = torch.from_numpy(rng.integers(0, max_pos, T).astype(np.int32)).cuda() if rot else None
    c["np"] = {n: (None if c[n] is None else to_f64(c[n])) for n in ("q", "k", "wq", "wk", "table")}
    c["np"]["pos"] = None if c["pos"] is None else c["pos"].cpu().numpy()
    return c


def _check_heads(got, x, w, table, pos, case):
    T, hq, hkv, D, rot, adjacent, norm, dtype, _ = case
    want = A.norm_rope(x, w, table, pos, rot, adjacent, norm, 1e-5)
    tol = (E if dtype == "bf16" else U) * np.abs(want) + (D + 16) * U * _magnitude(x, w, rot, adjacent, norm, 1e-5)
    err = np.abs(to_f64(got) - want)
    assert (err <= tol).all(), float((err - tol).max())


@pytest.mark.parametrize("case", HEADS)
def test_norm_rope(case):
    T, hq, hkv, D, rot, adjacent, norm, dtype, _ = case
    c, sffn = _heads_case(case), _mod()
    qo = torch.full((T, hq, D), math.nan, dtype=DT[dtype], device="cuda") if hq else None
    ko = torch.full((T, hkv, D), math.nan, dtype=DT[dtype], device="cuda") if hkv else None
    sffn.qk_norm_rope(c["h"], c["q"], c["k"], c["wq"], c["wk"], c["table"], c["pos"], qo, ko)
    n = c["np"]
    if hq:
        _check_heads(qo, n["q"], n["wq"], n["table"], n["pos"], case)
    if hkv:
        _check_heads(ko, n["k"], n["wk"], n["table"], n["pos"], case)


@pytest.mark.parametrize("case", HEADS)
def test_norm_rope_backward(case):
    T, hq, hkv, D, rot, adjacent, norm, dtype, _ = case
    c, sffn = _heads_case(case), _mod()
    rng = np.random.default_rng(9)
    gqo, gko = _randn(rng, (T, hq, D), dtype), _randn(rng, (T, hkv, D), dtype)
    # the gradients go into slices of one tensor, as the projection's backward reads them
    g = torch.full((T, hq + hkv + 1, D), math.nan, dtype=DT[dtype], device="cuda")
    gq, gk = g[:, :hq], g[:, hq:hq + hkv]
    gqw = torch.full((D,), math.nan, device="cuda")
    gkw = torch.full((D,), math.nan, device="cuda")
    ws = sffn.alloc_heads_workspace(c["h"])
    call = lambda: sffn.qk_norm_rope_bwd(  # noqa: E731
        c["h"], c["q"] if norm else None, c["k"] if norm else None, c["wq"], c["wk"], c["table"],
        c["pos"], gqo, gko, gq, gk, gqw, gkw, ws)
    call()
    assert torch.isnan(g[:, hq + hkv:]).all()  # nothing outside the slices
    n = c["np"]
    for x, w, gy, gx, gw, heads in ((n["q"], n["wq"], gqo, gq, gqw, hq),
                                    (n["k"], n["wk"], gko, gk, gkw, hkv)):
        if heads == 0:
            continue
        gy = to_f64(gy)
        want, want_w = A.norm_rope_backward(x, w, n["table"], n["pos"], gy, rot, adjacent, norm, 1e-5)
        # gn errs by 2 u of its pair; the mean of D products by (D + 16) u of
        # their absolute values; everything is scaled by r
        pair = _magnitude(gy, None, rot, adjacent, False, 0.0)
        if norm:
            r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-5)
            xh, wa = np.abs(x * r), 1.0 if w is None else np.abs(w)
            scale = r * (pair * wa + xh * (pair * wa * xh).mean(-1, keepdims=True))
            # the sums over tokens and heads: one wave's rows in sequence, then
            # blocks: at most T * heads additions
            tol_w = (D + 32 + T * heads) * U * (pair * xh).sum((0, 1))
            err_w = np.abs(to_f64(gw) - want_w)
            assert (err_w <= tol_w).all(), float((err_w - tol_w).max())
        else:
            scale = pair
        tol = (E if dtype == "bf16" else U) * np.abs(want) + 2 * (D + 32) * U * scale
        err = np.abs(to_f64(gx) - want)
        assert (err <= tol).all(), float((err - tol).max())
    if not norm:
        assert torch.isnan(gqw).all() and torch.isnan(gkw).all()
    else:
        first = [t.clone() for t in (gq, gk, gqw, gkw)]
        call()
        torch.cuda.synchronize()
        for a, b, live in zip(first, (gq, gk, gqw, gkw), (hq, hkv, hq, hkv)):
            assert not live or torch.equal(a, b)  # the same bits


def test_backward_against_differences():
    """The directional derivative of sum(gy * y) along a random direction, by
    central differences of the library's own float32 forward."""
    sffn = _mod()
    rng = np.random.default_rng(4)
    T, hq, hkv, D, rot = 6, 3, 2, 32, 24
    h = sffn.make_heads(T, hq, hkv, D, torch.float32, rot, 64, True, 1e-5)
    q, k, dq, dk = (_randn(rng, (T, n, D), "f32") for n in (hq, hkv, hq, hkv))
    wq, wk, dwq, dwk = (_randn(rng, (D,), "f32") for _ in range(4))
    gq_out, gk_out = _randn(rng, (T, hq, D), "f32"), _randn(rng, (T, hkv, D), "f32")
    pos = torch.from_numpy(rng.integers(0, 64, T).astype(np.int32)).cuda()
    tab = sffn.rotary_table(64, rot)

    def loss(s):
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        sffn.qk_norm_rope(h, q + s * dq, k + s * dk, wq + s * dwq, wk + s * dwk, tab, pos, qo, ko)
        return (qo.double() * gq_out.double()).sum().item() + (ko.double() * gk_out.double()).sum().item()

    gq, gk = torch.empty_like(q), torch.empty_like(k)
    gwq, gwk = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    sffn.qk_norm_rope_bwd(h, q, k, wq, wk, tab, pos, gq_out, gk_out, gq, gk, gwq, gwk,
                          sffn.alloc_heads_workspace(h))
    along = sum((a.double() * b.double()).sum().item()
                for a, b in ((gq, dq), (gk, dk), (gwq, dwq), (gwk, dwk)))
    s = 2.0 ** -7
    # the difference errs by s^2 / 6 of the third derivative (of the size of the
    # sum of |gy| over the elements) and by float32 rounding over s
    size = gq_out.abs().sum().item() + gk_out.abs().sum().item()
    assert abs((loss(s) - loss(-s)) / (2 * s) - along) <= size * (10 * s * s + 40 * U / s)


def test_position_outside_the_table_is_nan():
    sffn = _mod()
    rng = np.random.default_rng(5)
    h = sffn.make_heads(4, 2, 1, 64, torch.bfloat16, 32, 10, True)
    q, k = _randn(rng, (4, 2, 64), "bf16"), _randn(rng, (4, 1, 64), "bf16")
    pos = torch.tensor([0, 10, -1, 9], dtype=torch.int32, device="cuda")
    qo, ko = torch.zeros_like(q), torch.zeros_like(k)
    sffn.qk_norm_rope(h, q, k, None, None, sffn.rotary_table(10, 32), pos, qo, ko)
    for o in (qo, ko):
        bad = torch.isnan(o)
        assert bad[1:3, :, :32].all() and not bad[[0, 3]].any() and not bad[:, :, 32:].any()


# ---------------------------------------------------------------- the append
@pytest.mark.parametrize("T,hq,hkv,D,rot,norm,dtype,page,order", [
    (1, 8, 2, 128, 128, True, "bf16", 16, "token"),
    (70, 4, 4, 64, 64, True, "bf16", 1, "head"),     # head before token in memory
    (33, 0, 3, 80, 20, False, "f32", 24, "token"),   # no queries
    (2500, 5, 1, 128, 64, True, "bf16", 64, "head"),
])
def test_append(T, hq, hkv, D, rot, norm, dtype, page, order):
    sffn = _mod()
    rng = np.random.default_rng(T)
    n_pages = -(-T // page) + 4
    h = sffn.make_heads(T, hq, hkv, D, DT[dtype], rot, 4096, norm, 1e-5)
    qkv = _randn(rng, (T, hq + 2 * hkv, D), dtype)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    w = (1 + _randn(rng, (D,), "f32", 0.2)).to(DT[dtype]) if norm else None
    slots = rng.permutation(n_pages * page)[:T].astype(np.int32)
    slots[3::7] = -1
    if T > 20:
        slots[20] = n_pages * page      # past the cache: not stored
    pos = rng.integers(0, 4096, T).astype(np.int32)
    shape = (n_pages, page, hkv, D) if order == "token" else (n_pages, hkv, page, D)
    kc, vc = _randn(rng, shape, dtype), _randn(rng, shape, dtype)
    if order == "head":
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    k0, v0 = to_f64(kc), to_f64(vc)
    qo = torch.full((T, hq, D), math.nan, dtype=DT[dtype], device="cuda")
    tab = sffn.rotary_table(4096, rot)
    sffn.paged_kv_append(h, q, k, v, w, w, tab, torch.from_numpy(pos).cuda(),
                         torch.from_numpy(slots).cuda(), qo, kc, vc)
    wn, tn = None if w is None else to_f64(w), to_f64(tab)
    case = (T, hq, hkv, D, rot, False, norm, dtype, None)
    if hq:
        _check_heads(qo, to_f64(q), wn, tn, pos, case)
    want = A.paged_append(k0, A.norm_rope(to_f64(k), wn, tn, pos, rot, False, norm, 1e-5), slots)
    mag = A.paged_append(np.zeros_like(k0), _magnitude(to_f64(k), wn, rot, False, norm, 1e-5), slots)
    tol = ((E if dtype == "bf16" else U) * np.abs(want) + (D + 16) * U * mag) * (mag > 0)
    assert (np.abs(to_f64(kc) - want) <= tol).all()   # untouched rows: the same bits
    assert np.array_equal(to_f64(vc), A.paged_append(v0, to_f64(v), slots))


# ---------------------------------------------------------------- attention
def _attention_case(q_lens, kv_lens, hq, hkv, D, page, dtype, seed=0, scale=1.0, order="token"):
    rng = np.random.default_rng(seed)
    T, B = sum(q_lens), len(q_lens)
    pages = [-(-n // page) for n in kv_lens]
    n_pages, max_pages = sum(pages) + 2, max(pages + [1])
    bt = np.full((B, max_pages), -1, dtype=np.int32)   # entries that are not used
    perm, at = rng.permutation(n_pages), 0
    for b, n in enumerate(pages):
        bt[b, :n] = perm[at:at + n]
        at += n
    shape = (n_pages, page, hkv, D) if order == "token" else (n_pages, hkv, page, D)
    c = {"q": _randn(rng, (T, hq + 1, D), dtype, scale)[:, :hq], "k": _randn(rng, shape, dtype),
         "v": _randn(rng, shape, dtype), "bt": bt, "kv": np.array(kv_lens, dtype=np.int32),
         "qs": np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32), "page": page,
         "n_pages": n_pages, "dims": (T, B, hq, hkv, D), "dtype": dtype, "max_q": max(q_lens)}
    if order == "head":
        c["k"], c["v"] = c["k"].transpose(1, 2), c["v"].transpose(1, 2)
    # what lies behind a sequence's end must not matter: NaN and infinities
    for b, n in enumerate(kv_lens):
        if n % page:
            p = int(bt[b, n // page])
            c["k"][p, n % page:] = math.nan
            c["v"][p, n % page:] = math.nan
    for p in perm[at:]:
        c["k"][int(p)], c["v"][int(p)] = math.inf, math.nan
    return c


def _run(c, causal=True, window=0, sm_scale=None, max_q=None, max_kv=None, lse=True):
    sffn = _mod()
    T, B, hq, hkv, D = c["dims"]
    b = sffn.make_paged_batch(T, B, hq, hkv, D, DT[c["dtype"]], c["page"], c["n_pages"],
                              c["bt"].shape[1], max_q or c["max_q"],
                              int(c["kv"].max()) if max_kv is None else max_kv, causal, window,
                              sm_scale)
    out = torch.full((T, hq, D), 7.0, dtype=DT[c["dtype"]], device="cuda")
    ls = torch.full((T, hq), 7.0, device="cuda") if lse else None
    ws = sffn.alloc_paged_workspace(b)
    ws.fill_(255)   # NaN everywhere: no initial contents are needed
    dev = [torch.from_numpy(c[n]).cuda() for n in ("qs", "kv", "bt")]
    sffn.paged_attn_fwd(b, c["q"], c["k"], c["v"], *dev, out, ws, lse=ls)
    torch.cuda.synchronize()
    return out, ls


def _check_attention(c, out, lse, causal=True, window=0, sm_scale=None):
    T, B, hq, hkv, D = c["dims"]
    s = D ** -0.5 if sm_scale is None else sm_scale
    want, want_l, mag, smax = A.paged_attention(to_f64(c["q"]), to_f64(c["k"]), to_f64(c["v"]),
                                                c["qs"], c["kv"], c["bt"], s, causal, window)
    e = E if c["dtype"] == "bf16" else 0.0
    n = int(c["kv"].max())
    rel = 2 * ((D + 2) * smax + n + 64) * U + 2 * e
    own = (E if c["dtype"] == "bf16" else U)
    rows = np.arange(T) < c["qs"][-1]
    got, got_l = to_f64(out), to_f64(lse)
    assert (got[~rows] == 7.0).all() and (got_l[~rows] == 7.0).all()
    empty = np.isneginf(want_l) & rows[:, None]
    assert (got[empty] == 0).all() and np.isneginf(got_l[empty]).all()
    live = rows[:, None] & ~empty
    err = np.abs(got - want)[live]
    tol = (own * np.abs(want) + (1 + own) * rel[..., None] * mag)[live]
    assert (err <= tol).all(), (float(err.max()), float((err / np.maximum(tol, 1e-30)).max()))
    errl = np.abs(got_l[live] - want_l[live])
    toll = (rel + 4 * U * np.abs(want_l))[live]
    assert (errl <= toll).all(), (float(errl.max()), float((errl / toll).max()))
    if live.any() and not np.isnan(want[live]).any():
        fro = np.linalg.norm(got[live] - want[live]) / max(np.linalg.norm(want[live]), 1e-30)
        assert fro <= (5e-3 if c["dtype"] == "bf16" else 1e-5), fro


ATTENTION = [
    # q_lens, kv_lens, hq, hkv, D, page, dtype, causal, window, order
    ([1], [1], 1, 1, 128, 16, "bf16", True, 0, "token"),
    ([1], [129], 16, 4, 128, 16, "bf16", True, 0, "token"),
    ([1, 1, 1, 1], [1, 700, 64, 65], 32, 8, 128, 16, "bf16", True, 0, "token"),
    ([1] * 5, [33, 2000, 31, 32, 0], 8, 1, 64, 1, "bf16", True, 0, "token"),
    ([1, 1], [5000, 9], 28, 4, 128, 64, "bf16", True, 0, "head"),
    ([1, 1], [300, 511], 40, 1, 64, 24, "bf16", True, 0, "token"),     # 40 query heads on one
    ([3, 5, 1], [300, 1200, 77], 16, 4, 128, 16, "bf16", True, 0, "token"),
    ([4, 2], [900, 1300], 8, 2, 80, 7, "bf16", True, 100, "head"),
    ([64], [64], 4, 4, 128, 16, "bf16", True, 0, "token"),
    ([65, 1, 130], [65, 400, 1000], 8, 2, 128, 16, "bf16", True, 0, "token"),
    ([300], [300], 2, 1, 128, 64, "bf16", True, 0, "token"),
    ([257], [1500], 4, 2, 256, 32, "bf16", True, 0, "token"),
    ([200, 90], [200, 411], 3, 3, 64, 24, "bf16", True, 50, "token"),
    ([150], [150], 6, 2, 112, 16, "bf16", False, 0, "token"),
    ([40, 5], [100, 60], 4, 1, 8, 16, "bf16", False, 17, "token"),
    ([1, 0, 5, 0], [10, 5, 3, 0], 4, 2, 64, 4, "bf16", True, 0, "token"),  # more rows than keys
    ([70], [33], 4, 4, 96, 16, "bf16", True, 0, "token"),
    ([1, 1], [0, 0], 4, 4, 64, 16, "bf16", True, 0, "token"),
    ([1], [257], 8, 8, 80, 24, "f32", True, 0, "token"),
    ([1, 1], [1030, 3], 8, 1, 128, 16, "f32", True, 0, "head"),
    ([100, 1, 7], [300, 211, 90], 4, 2, 80, 24, "f32", True, 0, "token"),
    ([130], [130], 2, 2, 64, 16, "f32", True, 33, "token"),
    ([90], [200], 2, 1, 256, 16, "f32", False, 0, "token"),
    ([9, 20], [5, 50], 2, 2, 32, 5, "f32", True, 3, "token"),
]


@pytest.mark.parametrize("q_lens,kv_lens,hq,hkv,D,page,dtype,causal,window,order", ATTENTION)
def test_attention(q_lens, kv_lens, hq, hkv, D, page, dtype, causal, window, order):
    c = _attention_case(q_lens, kv_lens, hq, hkv, D, page, dtype, order=order)
    out, lse = _run(c, causal, window)
    _check_attention(c, out, lse, causal, window)
    # the same bits again, also without lse and with looser bounds of the lengths
    again, _ = _run(c, causal, window, lse=False)
    assert torch.equal(out, again)


MORE = [
    # many splits, and a split range that ends inside a chunk
    ([1], [9001], 4, 1, 128, 16, "bf16", True, 0, "token"),
    ([2, 1], [7000, 3000], 6, 2, 256, 8, "bf16", True, 0, "head"),
    ([1, 3], [2500, 1111], 4, 4, 64, 24, "f32", True, 0, "token"),
    ([1], [1500], 2, 1, 256, 32, "f32", True, 0, "token"),
    # chunks over long ranges: row tiles whose keys are split, with and without a window
    ([100], [3000], 4, 2, 128, 16, "bf16", True, 0, "token"),
    ([90, 40], [2800, 1900], 4, 1, 64, 7, "bf16", True, 700, "token"),
    ([130], [2000], 3, 1, 96, 16, "bf16", False, 900, "token"),
    ([70], [1300], 2, 2, 128, 1, "f32", True, 500, "head"),
    # windows for few rows, split and not
    ([4, 1, 3], [5000, 900, 2100], 8, 2, 128, 16, "bf16", True, 1500, "token"),
    ([7, 2], [400, 800], 8, 1, 64, 16, "bf16", False, 60, "token"),
    # group sizes that divide no tile, and 33 to 64 rows (two tiles of few rows)
    ([9, 5, 1], [900, 30, 2000], 7, 1, 128, 16, "bf16", True, 0, "token"),
    ([13, 200], [700, 1000], 15, 3, 80, 16, "bf16", True, 0, "token"),
    ([3], [50], 66, 1, 64, 16, "bf16", True, 0, "token"),
    ([2, 1], [300, 70], 100, 1, 32, 16, "f32", True, 0, "token"),
]


@pytest.mark.parametrize("q_lens,kv_lens,hq,hkv,D,page,dtype,causal,window,order", MORE)
def test_attention_splits_and_groups(q_lens, kv_lens, hq, hkv, D, page, dtype, causal, window, order):
    test_attention(q_lens, kv_lens, hq, hkv, D, page, dtype, causal, window, order)


FEW_AND_MANY_ROWS = [
    # rows around one and two tiles of few rows, with and without longer sequences beside
    # them: 32, 33 .. 64 and 65 rows of a sequence
    ([8, 9, 16, 17, 1], [300, 90, 700, 130, 2000], 8, 2, 128, 16, 0),
    ([8, 9, 16, 1], [300, 90, 700, 2000], 8, 2, 128, 16, 0),
    ([32, 33, 64, 65, 1, 0], [40, 900, 64, 65, 3, 9], 3, 3, 64, 24, 0),
    ([16, 17, 33], [1500, 1400, 33], 4, 2, 80, 1, 70),
    # a single token has more rows than one tile, or than two
    ([1, 2, 30], [500, 40, 300], 48, 1, 64, 16, 0),
    ([1, 1], [1200, 7], 48, 1, 128, 8, 0),
    ([1, 5, 1], [900, 5, 0], 130, 2, 64, 16, 0),
]


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
    c = _attention_case(q_lens, kv_lens, 8, 2, 64, 16, dtype, seed=n_seqs)
    out, lse = _run(c)
    _check_attention(c, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_padding_rows_are_left_alone(dtype):
    """Rows of q past the last sequence, as in a batch padded to a fixed size."""
    c = _attention_case([3, 80, 30], [100, 90, 50], 4, 2, 64, 16, dtype, seed=21)
    c["qs"], c["kv"], c["bt"] = c["qs"][:3].copy(), c["kv"][:2].copy(), c["bt"][:2].copy()
    T, B, hq, hkv, D = c["dims"]
    c["dims"] = (T, 2, hq, hkv, D)
    out, lse = _run(c)
    _check_attention(c, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_wrong_lengths_and_pages_stay_in_bounds(dtype):
    """Lengths beyond the stated bounds, rows out of range and pages that do not exist
    are cut to the bounds (so nothing outside the buffers is touched), and the
    sequences beside them come out right."""
    lens = ([1, 1, 40, 1, 90], [200, 64, 300, 90, 150])
    c = _attention_case(*lens, 4, 2, 64, 16, dtype, seed=22)
    T, B, hq, hkv, D = c["dims"]
    good, good_l = _run(c)
    bad = dict(c, kv=c["kv"].copy(), qs=c["qs"].copy(), bt=c["bt"].copy())
    bad["kv"][1] = 1 << 30
    bad["kv"][3] = -5
    bad["bt"][2, :3] = [1 << 30, -7, c["n_pages"]]
    out, lse = _run(bad, max_kv=300)
    keep = [i for b in (0, 4) for i in range(c["qs"][b], c["qs"][b + 1])]
    assert torch.equal(out[keep], good[keep]) and torch.equal(lse[keep], good_l[keep])
    # the sequence of negative length is empty
    empty = int(c["qs"][3])
    assert (out[empty] == 0).all() and torch.isneginf(lse[empty]).all()
    # rows out of range: the last sequence starts before its neighbour ends
    bad = dict(c, qs=c["qs"].copy())
    bad["qs"][1:] = [-3, 1 << 30, 10, 43, 2000]
    _run(bad, max_q=90)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("max_q,max_kv", [(100, 512), (1000, 100 * 16)])
def test_bounds_of_the_lengths_are_upper_bounds(dtype, max_q, max_kv):
    c = _attention_case([1, 40, 3], [500, 300, 512], 4, 2, 64, 16, dtype, seed=3)
    c["bt"] = np.concatenate([c["bt"], np.full((3, 100 - c["bt"].shape[1]), -5, np.int32)], 1)
    out, lse = _run(c, max_q=max_q, max_kv=max_kv)
    _check_attention(c, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_len", [1, 8, 150])
def test_large_scores(dtype, q_len):
    """Scores of several hundred: the running maximum keeps the sums finite."""
    c = _attention_case([q_len], [700], 4, 2, 64, 16, dtype, seed=5, scale=40.0)
    out, lse = _run(c, sm_scale=0.3)
    _check_attention(c, out, lse, sm_scale=0.3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("sm_scale", [0.0, -0.2])
def test_zero_and_negative_scale(dtype, sm_scale):
    c = _attention_case([1, 70], [90, 130], 4, 2, 64, 16, dtype, seed=6)
    out, lse = _run(c, sm_scale=sm_scale)
    _check_attention(c, out, lse, sm_scale=sm_scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_len", [4, 100])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_later_keys_do_not_reach_earlier_rows(dtype, q_len, bad):
    """NaN or infinity in a key and a value that only the last rows see: the rows
    before it come out as without it."""
    c = _attention_case([q_len], [q_len + 60], 4, 2, 64, 16, dtype, seed=7)
    clean, clean_l = _run(c)
    j = q_len + 60 - 2                       # seen by the last two rows
    page = int(c["bt"][0, j // 16])
    c["v"][page, j % 16, :, 3::5] = bad
    c["k"][page, j % 16, 1] = bad
    out, lse = _run(c)
    assert torch.equal(out[:-2], clean[:-2]) and torch.equal(lse[:-2], clean_l[:-2])
    assert not torch.isfinite(out[-2:, :, 3::5]).any()
    assert torch.isfinite(out[-2:, :2, 0:3]).all()    # head 0 has finite keys


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_before_the_window_are_not_used(dtype):
    """Pages wholly before the window may be gone from the table, and rows before
    it in its first page may hold anything."""
    c = _attention_case([3, 1], [500, 400], 4, 2, 64, 16, dtype, seed=8)
    out, lse = _run(c, window=100)
    _check_attention(c, out, lse, window=100)
    for b, (nq, n) in enumerate(((3, 500), (1, 400))):
        lo = n - nq - 100 + 1
        for j in range(lo):
            p = int(c["bt"][b, j // 16])
            c["k"][p, j % 16], c["v"][p, j % 16] = math.nan, math.nan
        c["bt"][b, :lo // 16] = -1
    again, again_l = _run(c, window=100)
    assert torch.equal(out, again) and torch.equal(lse, again_l)


def test_on_a_side_stream_and_in_a_graph():
    """Captured once and replayed with changing lengths and eager work between."""
    sffn = _mod()
    c = _attention_case([1, 1, 1], [900, 40, 300], 8, 2, 128, 16, "bf16", seed=11)
    T, B, hq, hkv, D = c["dims"]
    b = sffn.make_paged_batch(T, B, hq, hkv, D, torch.bfloat16, 16, c["n_pages"], c["bt"].shape[1], 1, 900)
    ws = sffn.alloc_paged_workspace(b)
    out, lse = torch.empty((T, hq, D), dtype=torch.bfloat16, device="cuda"), torch.empty((T, hq), device="cuda")
    qs, kv, bt = (torch.from_numpy(c[n]).cuda() for n in ("qs", "kv", "bt"))
    q = c["q"].contiguous()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sffn.paged_attn_fwd(b, q, c["k"], c["v"], qs, kv, bt, out, ws, lse=lse)
    torch.cuda.current_stream().wait_stream(side)
    c["q"] = q
    _check_attention(c, out, lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sffn.paged_attn_fwd(b, q, c["k"], c["v"], qs, kv, bt, out, ws, lse=lse)
    for i, lens in enumerate(([900, 40, 300], [1, 33, 299], [555, 2, 150], [900, 40, 300])):
        c["kv"] = np.array(lens, dtype=np.int32)
        kv.copy_(torch.from_numpy(c["kv"]))
        q.normal_()
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        _check_attention(c, out, lse)


def test_cache_beyond_four_gib():
    """Byte offsets past 32 bits, both in the append and in the attention."""
    sffn = _mod()
    page, hkv, D = 64, 8, 256
    n_pages = (5 << 30) // (page * hkv * D * 2)
    kc = torch.empty((n_pages, page, hkv, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    rng = np.random.default_rng(12)
    T = 100
    qkv = _randn(rng, (T, 3 * hkv, D), "bf16")
    q, k, v = qkv[:, :hkv], qkv[:, hkv:2 * hkv], qkv[:, 2 * hkv:]
    pages = np.array([n_pages - 1, n_pages // 2 + 3], dtype=np.int32)
    slots = (pages[np.arange(T) // page] * page + np.arange(T) % page).astype(np.int32)
    h = sffn.make_heads(T, hkv, hkv, D, torch.bfloat16)
    qo = torch.empty((T, hkv, D), dtype=torch.bfloat16, device="cuda")
    sffn.paged_kv_append(h, q, k, v, None, None, None, None, torch.from_numpy(slots).cuda(), qo, kc, vc)
    assert torch.equal(kc.view(-1, hkv, D)[torch.from_numpy(slots).cuda().long()], k)
    small = {"q": q, "k": kc[torch.from_numpy(pages).cuda().long()], "v": vc[torch.from_numpy(pages).cuda().long()],
             "bt": np.array([[0, 1]], np.int32), "kv": np.array([T], np.int32), "qs": np.array([0, T], np.int32),
             "page": page, "n_pages": 2, "dims": (T, 1, hkv, hkv, D), "dtype": "bf16", "max_q": T}
    big = dict(small, k=kc, v=vc, bt=pages[None, :].copy(), n_pages=n_pages)
    o1, l1 = _run(small)
    o2, l2 = _run(big)
    assert torch.equal(o1, o2) and torch.equal(l1, l2)
    _check_attention(small, o1, l1)
