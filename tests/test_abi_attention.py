"""Refusals of the attention side's entry points, on the host: reported before
anything is launched (no GPU needed)."""
from __future__ import annotations

import ctypes

import pytest
import torch

ARG, UNSUPPORTED, WORKSPACE, OK = -1, -2, -3, 0
P = 0x10000          # aligned fake device pointers: never dereferenced
ODD = 0x10008        # 8-byte aligned
ODD2 = 0x10002


@pytest.fixture(scope="module")
def sffn():
    import os
    from activation_sparse_feed_amd import build
    if not os.path.exists(build.LIB):
        build.build()
    from activation_sparse_feed_amd import sffn as mod
    return mod


def heads(sffn, **kw):
    h = sffn.make_heads(8, 4, 2, 64, torch.bfloat16, 32, 100, True)
    for k, v in kw.items():
        setattr(h, k, v)
    return h


BAD_HEADS = [
    (dict(T=-1), ARG), (dict(n_q_heads=-1), ARG), (dict(n_kv_heads=-1), ARG), (dict(head_dim=0), ARG),
    (dict(head_dim=60), UNSUPPORTED), (dict(head_dim=264), UNSUPPORTED), (dict(rot_dim=-4), ARG),
    (dict(rot_dim=68), ARG), (dict(rot_dim=6), UNSUPPORTED), (dict(max_pos=0), ARG), (dict(max_pos=-1), ARG),
    (dict(norm=2), ARG), (dict(rot_adjacent=-1), ARG), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG),
    (dict(eps=float("inf")), ARG), (dict(dtype=7), ARG), (dict(n_q_heads=5000), UNSUPPORTED),
]
ROWS = (P, 512, 64)


def norm_rope(sffn, h, q=ROWS, k=ROWS, wq=P, wk=P, table=P, pos=P, qo=ROWS, ko=ROWS):
    return sffn._lib.qk_norm_rope(h, *q, *k, wq, wk, table, pos, *qo, *ko, None)


def norm_rope_bwd(sffn, h, q=ROWS, k=ROWS, wq=P, wk=P, table=P, pos=P, gqo=ROWS, gko=ROWS, gq=ROWS,
                  gk=ROWS, gwq=P, gwk=P, ws=P, ws_n=1 << 30):
    return sffn._lib.qk_norm_rope_bwd(h, *q, *k, wq, wk, table, pos, *gqo, *gko, *gq, *gk, gwq, gwk,
                                      ws, ws_n, None)


CACHE = (P, 16 * 128, 128, 64)


def append(sffn, h, q=ROWS, k=ROWS, v=ROWS, table=P, pos=P, slots=P, qo=ROWS, kc=CACHE, vc=CACHE,
           n_pages=4, page=16):
    return sffn._lib.paged_kv_append(h, *q, *k, *v, None, None, table, pos, slots, *qo, *kc, *vc,
                                     n_pages, page, None)


@pytest.mark.parametrize("kw,status", BAD_HEADS)
def test_bad_heads(sffn, kw, status):
    h = heads(sffn, **kw)
    assert norm_rope(sffn, h) == status
    assert norm_rope_bwd(sffn, h) == status
    assert append(sffn, h) == status
    assert sffn._lib.qk_norm_rope_bwd_workspace_bytes(h) == 0


def test_no_struct(sffn):
    assert norm_rope(sffn, None) == ARG and norm_rope_bwd(sffn, None) == ARG
    assert append(sffn, None) == ARG and attn(sffn, None) == ARG


BAD_ROWS = [((None, 512, 64), ARG), ((ODD, 512, 64), ARG), ((P, -512, 64), ARG),
            ((P, 512, 68), UNSUPPORTED), ((P, 516, 64), UNSUPPORTED)]
BAD_OUT = BAD_ROWS + [((P, 0, 64), ARG), ((P, 512, 0), ARG), ((P, 512, 56), ARG)]


@pytest.mark.parametrize("rows,status", BAD_OUT)
def test_bad_rows(sffn, rows, status):
    h = heads(sffn)
    for name in ("qo", "ko"):
        assert norm_rope(sffn, h, **{name: rows}) == status
    for name in ("gq", "gk"):
        assert norm_rope_bwd(sffn, h, **{name: rows}) == status
    assert append(sffn, h, qo=rows) == status
    if (rows, status) in BAD_ROWS:  # an input's rows may overlap
        for name in ("q", "k"):
            assert norm_rope(sffn, h, **{name: rows}) == status
            assert norm_rope_bwd(sffn, h, **{name: rows}) == status
        for name in ("gqo", "gko"):
            assert norm_rope_bwd(sffn, h, **{name: rows}) == status
        for name in ("q", "k", "v"):
            assert append(sffn, h, **{name: rows}) == status


def test_arrays_and_workspace(sffn):
    h = heads(sffn)
    for call in (norm_rope, norm_rope_bwd, append):
        assert call(sffn, h, table=None) == ARG and call(sffn, h, pos=None) == ARG
        assert call(sffn, h, table=ODD2) == ARG and call(sffn, h, pos=ODD2) == ARG
    assert norm_rope(sffn, h, wq=ODD) == ARG and norm_rope_bwd(sffn, h, wk=ODD) == ARG
    assert norm_rope_bwd(sffn, h, gwq=ODD2) == ARG
    assert append(sffn, h, slots=None) == ARG and append(sffn, h, slots=ODD2) == ARG
    need = sffn._lib.qk_norm_rope_bwd_workspace_bytes(h)
    assert need >= 2 * 64 * 4
    assert norm_rope_bwd(sffn, h, ws_n=need - 1) == WORKSPACE
    assert norm_rope_bwd(sffn, h, ws=None) == WORKSPACE and norm_rope_bwd(sffn, h, ws=ODD) == WORKSPACE
    assert sffn._lib.qk_norm_rope_bwd_workspace_bytes(heads(sffn, norm=0)) == 0


def test_bad_cache(sffn):
    h = heads(sffn)
    for c, status in (((None, 2048, 128, 64), ARG), ((ODD, 2048, 128, 64), ARG), ((P, 0, 128, 64), ARG),
                      ((P, 2048, 0, 64), ARG), ((P, 2048, 128, 0), ARG), ((P, 2052, 128, 64), UNSUPPORTED),
                      ((P, 2048, 132, 64), UNSUPPORTED), ((P, 2048, 128, 68), UNSUPPORTED)):
        assert append(sffn, h, kc=c) == status and append(sffn, h, vc=c) == status
        assert attn(sffn, batch(sffn), kc=c) == status and attn(sffn, batch(sffn), vc=c) == status
    assert append(sffn, h, n_pages=-1) == ARG and append(sffn, h, page=0) == ARG
    assert append(sffn, heads(sffn, n_kv_heads=0)) == ARG


def test_nothing_to_do_needs_no_buffers(sffn):
    none, nocache = (None, 0, 0), (None, 0, 0, 0)
    h = heads(sffn, T=0)
    assert norm_rope(sffn, h, none, none, None, None, None, None, none, none) == OK
    assert append(sffn, h, none, none, none, None, None, None, none, nocache, nocache) == OK
    h = heads(sffn, n_q_heads=0, n_kv_heads=0)
    assert norm_rope(sffn, h, none, none, None, None, None, None, none, none) == OK
    h = heads(sffn, T=0, norm=0)
    assert norm_rope_bwd(sffn, h, none, none, None, None, None, None, none, none, none, none, None,
                         None, None, 0) == OK
    for kw in (dict(T=0), dict(n_seqs=0), dict(max_q=0)):
        assert attn(sffn, batch(sffn, **kw), none, nocache, nocache, None, None, None, none, None,
                    None, 0) == OK


def batch(sffn, **kw):
    b = sffn.make_paged_batch(8, 2, 4, 2, 64, torch.bfloat16, 16, 4, 100, 4, 1600)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


def attn(sffn, b, q=ROWS, kc=CACHE, vc=CACHE, qs=P, kv=P, bt=P, out=ROWS, lse=P, ws=P, ws_n=1 << 40):
    return sffn._lib.paged_attn_fwd(b, *q, *kc, *vc, qs, kv, bt, *out, lse, ws, ws_n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), ARG), (dict(n_seqs=-1), ARG), (dict(n_q_heads=0), ARG), (dict(n_kv_heads=0), ARG),
    (dict(n_q_heads=3), ARG), (dict(head_dim=0), ARG), (dict(head_dim=12), UNSUPPORTED),
    (dict(head_dim=512), UNSUPPORTED), (dict(page_size=0), ARG), (dict(n_pages=-1), ARG),
    (dict(n_pages=0), ARG), (dict(max_pages=99), ARG), (dict(max_pages=-1), ARG), (dict(max_q=-1), ARG),
    (dict(max_kv=-1), ARG), (dict(max_kv=1601), ARG), (dict(causal=2), ARG), (dict(window=-1), ARG),
    (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG), (dict(dtype=2), ARG),
    (dict(T=1 << 29), UNSUPPORTED), (dict(n_seqs=(1 << 20) + 1), UNSUPPORTED),
    (dict(max_pages=1 << 27, max_kv=(1 << 30) + 1), UNSUPPORTED),
])
def test_bad_batch(sffn, kw, status):
    b = batch(sffn, **kw)
    assert attn(sffn, b) == status
    assert sffn._lib.paged_attn_workspace_bytes(b) == 0


def test_attention_arguments(sffn):
    b = batch(sffn)
    for rows, status in BAD_ROWS:
        assert attn(sffn, b, q=rows) == status
    for rows, status in BAD_OUT:
        assert attn(sffn, b, out=rows) == status
    for name in ("qs", "kv", "bt"):
        assert attn(sffn, b, **{name: None}) == ARG and attn(sffn, b, **{name: ODD2}) == ARG
    assert attn(sffn, b, lse=ODD2) == ARG
    need = sffn._lib.paged_attn_workspace_bytes(b)
    assert need > 0      # 1600 keys are split
    assert attn(sffn, b, ws_n=need - 1) == WORKSPACE
    assert attn(sffn, b, ws=None) == WORKSPACE and attn(sffn, b, ws=ODD) == WORKSPACE


def test_workspace_stays_small(sffn):
    """The splits' partial results: a few MiB for a step of single tokens, none for
    a long prompt."""
    def need(T, n_seqs, max_q, max_kv):
        return sffn.paged_attn_workspace_bytes(sffn.make_paged_batch(
            T, n_seqs, 32, 8, 128, torch.bfloat16, 16, 1 << 20, 1 << 16, max_q, max_kv))
    assert need(16384, 1, 16384, 16384) == 0
    assert 0 < need(32, 32, 1, 4096) <= 64 << 20
    assert need(1, 1, 1, 1 << 20) <= 64 << 20


def test_binding_checks(sffn):
    """Shapes, types and devices are checked before the library is called."""
    h = heads(sffn)
    q = torch.zeros((8, 4, 64), dtype=torch.bfloat16)
    k = torch.zeros((8, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="q must be"):
        sffn.qk_norm_rope(h, q[:, :3], k, None, None, None, None, q, k)
    with pytest.raises(TypeError, match="q must be"):
        sffn.qk_norm_rope(h, q.float(), k, None, None, None, None, q, k)
    with pytest.raises(ValueError, match="GPU"):
        sffn.qk_norm_rope(h, q, k, None, None, None, None, q, k)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        sffn.make_heads(1, 1, 1, 64, torch.float16)
    with pytest.raises(ValueError, match="k_cache must be"):
        sffn.paged_attn_fwd(batch(sffn), _gpu_like(q), k, k, None, None, None, q, None)


class _gpu_like:
    """A CPU tensor's shape, type and strides with a GPU's flag."""

    def __init__(self, t):
        self.t, self.shape, self.dtype, self.is_cuda = t, t.shape, t.dtype, True

    def stride(self):
        return self.t.stride()

    def data_ptr(self):
        return self.t.data_ptr()


def test_struct_layouts(sffn):
    assert ctypes.sizeof(sffn.Heads) == 40 and ctypes.sizeof(sffn.PagedBatch) == 56


def test_rotary_table(sffn):
    t = sffn.rotary_table(5, 8, device="cpu")
    assert t.shape == (5, 8) and t.dtype == torch.float32
    assert torch.equal(t[0], torch.tensor([1.0] * 4 + [0.0] * 4))
    assert torch.allclose(t[3, 1], torch.cos(torch.tensor(3 * 0.1))) and torch.allclose(
        t[3, 5], torch.sin(torch.tensor(3 * 0.1)))


def test_paged_slots(sffn):
    bt = torch.tensor([[4, 2, 7], [1, 0, 3]], dtype=torch.int32)
    seq, pos = torch.tensor([0, 0, 1, 1]), torch.tensor([0, 9, 5, 14])
    assert sffn.paged_slots(bt, seq, pos, 5).tolist() == [20, 14, 0, 19]
