"""Refusals of the 4-bit cache's entry points, on the host: reported before anything is
launched (no GPU needed)."""
from __future__ import annotations

import ctypes

import pytest
import torch

from test_abi_attention import (ARG, BAD_HEADS, BAD_OUT, BAD_ROWS, ODD, ODD2, OK, P, ROWS, UNSUPPORTED,
                                WORKSPACE, batch, heads, sffn)  # noqa: F401
from test_attention_binding import OnGpu, _NoStream, gpu

NONE = (None, 512, 64)
# 4 pages of 16 tokens, 2 heads of 64: 32 bytes of codes, 2 of scales
CODES, SCALES = (16 * 64, 32, 16 * 32), (16 * 4, 2, 32)


def rows4(sffn, codes=P, scales=P, c=CODES, s=SCALES):  # noqa: F811
    return sffn.Mx4Rows(codes, scales, *c, *s)


def append(sffn, h, q=ROWS, k=ROWS, v=ROWS, table=P, pos=P, slots=P, qo=ROWS, kc=..., vc=..., n_pages=4,  # noqa: F811
           page=16, w=None):
    kc = rows4(sffn) if kc is ... else kc
    vc = rows4(sffn) if vc is ... else vc
    return sffn._lib.paged_kv_append_mx4(h, *q, *k, *v, w, w, table, pos, slots, *qo, kc, vc, n_pages,
                                         page, None)


def read(sffn, T=8, heads=2, dim=64, dtype=1, kc=..., vc=..., n_pages=4, page=16, slots=P, ko=ROWS, vo=ROWS):  # noqa: F811
    kc = rows4(sffn) if kc is ... else kc
    vc = rows4(sffn) if vc is ... else vc
    return sffn._lib.paged_kv_read_mx4(T, heads, dim, dtype, kc, vc, n_pages, page, slots, *ko, *vo, None)


def attn(sffn, b, q=ROWS, kc=..., vc=..., qs=P, kv=P, bt=P, out=ROWS, lse=P, ws=P, ws_n=1 << 40):  # noqa: F811
    kc = rows4(sffn) if kc is ... else kc
    vc = rows4(sffn) if vc is ... else vc
    return sffn._lib.paged_attn_mx4_fwd(b, *q, kc, vc, qs, kv, bt, *out, lse, ws, ws_n, None)


@pytest.mark.parametrize("kw,status", BAD_HEADS)
def test_bad_heads(sffn, kw, status):  # noqa: F811
    assert append(sffn, heads(sffn, **kw)) == status


def test_no_struct(sffn):  # noqa: F811
    assert append(sffn, None) == ARG and attn(sffn, None) == ARG
    h, b = heads(sffn), batch(sffn)
    for kw in (dict(kc=None), dict(vc=None)):
        assert append(sffn, h, **kw) == ARG and attn(sffn, b, **kw) == ARG and read(sffn, **kw) == ARG


@pytest.mark.parametrize("rows,status", BAD_OUT)
def test_bad_rows(sffn, rows, status):  # noqa: F811
    h, b = heads(sffn), batch(sffn)
    assert append(sffn, h, qo=rows) == status and attn(sffn, b, out=rows) == status
    if rows[0] is not None:      # None: not read
        assert read(sffn, ko=rows) == status and read(sffn, vo=rows) == status
    if (rows, status) in BAD_ROWS:  # an input's rows may overlap
        for name in ("q", "k", "v"):
            assert append(sffn, h, **{name: rows}) == status
        assert attn(sffn, b, q=rows) == status


@pytest.mark.parametrize("kw,status", [
    (dict(codes=None), ARG), (dict(scales=None), ARG), (dict(codes=ODD2), ARG),
    (dict(c=(0, 32, 512)), ARG), (dict(c=(1024, 28, 512)), ARG), (dict(c=(1024, 32, -512)), ARG),
    (dict(s=(1, 2, 32)), ARG), (dict(s=(64, 1, 32)), ARG), (dict(s=(64, 2, 0)), ARG),
    (dict(c=(1026, 32, 512)), UNSUPPORTED), (dict(c=(1024, 33, 512)), UNSUPPORTED),
    (dict(c=(1024, 32, 514)), UNSUPPORTED),
])
def test_bad_cache(sffn, kw, status):  # noqa: F811
    c = rows4(sffn, **kw)
    for name in ("kc", "vc"):
        assert append(sffn, heads(sffn), **{name: c}) == status
        assert attn(sffn, batch(sffn), **{name: c}) == status
        assert read(sffn, **{name: c}) == status


def test_strides_of_single_dimensions_are_not_looked_at(sffn):  # noqa: F811
    """One page, one token, one head: any strides; what is refused next is a missing buffer."""
    c = rows4(sffn, c=(0, 0, 0), s=(0, 0, 0))
    assert append(sffn, heads(sffn, n_q_heads=1, n_kv_heads=1), kc=c, vc=c, n_pages=1, page=1,
                  slots=None) == ARG
    assert read(sffn, heads=1, kc=c, vc=c, n_pages=1, page=1, slots=None) == ARG
    odd = rows4(sffn, codes=P + 4, scales=P + 1)      # codes by words of 4 bytes, scales by bytes
    assert append(sffn, heads(sffn), kc=odd, vc=odd, slots=None) == ARG


def test_arrays_and_sizes(sffn):  # noqa: F811
    h = heads(sffn)
    for kw in (dict(table=None), dict(pos=None), dict(table=ODD2), dict(pos=ODD2), dict(slots=None),
               dict(slots=ODD2), dict(w=ODD), dict(n_pages=-1), dict(page=0)):
        assert append(sffn, h, **kw) == ARG
    assert append(sffn, heads(sffn, n_kv_heads=0)) == ARG
    for kw, status in ((dict(T=-1), ARG), (dict(heads=0), ARG), (dict(dim=0), ARG), (dict(dtype=2), ARG),
                       (dict(dim=60), UNSUPPORTED), (dict(dim=264), UNSUPPORTED), (dict(heads=4097), UNSUPPORTED),
                       (dict(n_pages=-1), ARG), (dict(page=0), ARG), (dict(slots=None), ARG),
                       (dict(slots=ODD2), ARG)):
        assert read(sffn, **kw) == status


def test_sizes_that_no_launch_takes(sffn):  # noqa: F811
    for T, status in (((1 << 26) - 4, ARG), ((1 << 26) - 3, UNSUPPORTED), ((1 << 31) - 1, UNSUPPORTED)):
        assert append(sffn, heads(sffn, T=T), q=NONE) == status
    for T, status in (((1 << 26) - 32, ARG), ((1 << 26) - 31, UNSUPPORTED), ((1 << 31) - 1, UNSUPPORTED)):
        assert read(sffn, T=T, slots=None) == status
    # a slot has 32 bits
    assert append(sffn, heads(sffn), q=NONE, n_pages=1 << 27) == ARG
    assert append(sffn, heads(sffn), q=NONE, n_pages=(1 << 27) + 1) == UNSUPPORTED
    assert read(sffn, slots=None, n_pages=1 << 27) == ARG
    assert read(sffn, slots=None, n_pages=(1 << 27) + 1) == UNSUPPORTED


def test_nothing_to_do_needs_no_buffers(sffn):  # noqa: F811
    none = (None, 0, 0)
    assert append(sffn, heads(sffn, T=0), none, none, none, None, None, None, none, None, None) == OK
    assert read(sffn, T=0, kc=None, vc=None, slots=None, ko=none, vo=none) == OK
    assert read(sffn, kc=None, vc=None, slots=None, ko=none, vo=none) == OK
    for kw in (dict(T=0), dict(n_seqs=0), dict(max_q=0)):
        assert attn(sffn, batch(sffn, **kw), none, None, None, None, None, None, none, None, None, 0) == OK
    # a batch without keys needs no cache: what is refused next is a missing buffer
    assert attn(sffn, batch(sffn, max_kv=0, n_pages=0), out=NONE, kc=None, vc=None, bt=None) == ARG


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), ARG), (dict(n_q_heads=3), ARG), (dict(head_dim=12), UNSUPPORTED), (dict(head_dim=512), UNSUPPORTED),
    (dict(page_size=0), ARG), (dict(n_pages=0), ARG), (dict(max_pages=99), ARG), (dict(max_kv=1601), ARG),
    (dict(causal=2), ARG), (dict(window=-1), ARG), (dict(scale=float("nan")), ARG), (dict(dtype=2), ARG),
    (dict(T=1 << 29), UNSUPPORTED), (dict(n_seqs=(1 << 20) + 1), UNSUPPORTED),
    (dict(max_pages=1 << 27, max_kv=(1 << 30) + 1), UNSUPPORTED),
])
def test_bad_batch(sffn, kw, status):  # noqa: F811
    b = batch(sffn, **kw)
    assert attn(sffn, b) == status
    assert sffn._lib.paged_attn_mx4_workspace_bytes(b) == 0


def test_attention_arguments(sffn):  # noqa: F811
    b = batch(sffn)
    for name in ("qs", "kv", "bt"):
        assert attn(sffn, b, **{name: None}) == ARG and attn(sffn, b, **{name: ODD2}) == ARG
    assert attn(sffn, b, lse=ODD2) == ARG
    need = sffn._lib.paged_attn_mx4_workspace_bytes(b)
    assert need > 0      # 1600 keys are split
    assert attn(sffn, b, ws_n=need - 1) == WORKSPACE
    assert attn(sffn, b, ws=None) == WORKSPACE and attn(sffn, b, ws=ODD) == WORKSPACE


@pytest.mark.parametrize("kw,status", [
    # single tokens: workgroups of four waves (1600 keys) or eight, 2^32 threads are too many
    (dict(n_seqs=1 << 20, n_q_heads=16, n_kv_heads=16), UNSUPPORTED),
    (dict(n_seqs=(1 << 20) - 1, n_q_heads=16, n_kv_heads=16), ARG),
    (dict(n_seqs=1 << 20, n_q_heads=8, n_kv_heads=8, max_kv=1000), UNSUPPORTED),
    (dict(n_seqs=(1 << 20) - 1, n_q_heads=8, n_kv_heads=8, max_kv=1000), ARG),
    (dict(n_seqs=1 << 20, n_q_heads=4096, n_kv_heads=4096), UNSUPPORTED),
    (dict(T=1 << 18, max_q=1000, n_seqs=1 << 18, n_q_heads=4096, n_kv_heads=4096), UNSUPPORTED),
    (dict(T=5000, max_q=1000, n_seqs=1 << 12, n_q_heads=64, n_kv_heads=8), ARG),
    (dict(T=1 << 18, max_q=65, n_seqs=1 << 18, n_q_heads=4096, n_kv_heads=4096, max_kv=0), UNSUPPORTED),
])
def test_grids_of_the_attention(sffn, kw, status):  # noqa: F811
    b = batch(sffn, **kw)
    assert attn(sffn, b, q=NONE) == status
    if status != ARG:
        assert sffn._lib.paged_attn_mx4_workspace_bytes(b) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("max_q", [1, 8, 16, 500])
@pytest.mark.parametrize("window", [0, 5000])
def test_workspace_under_the_limits_of_a_model(sffn, dtype, dim, max_q, window):  # noqa: F811
    for n_seqs in (1, 32, 256, 10000):
        for max_kv in (4096, 131072, 1 << 20):
            b = sffn.make_paged_batch(n_seqs * max_q, n_seqs, 32, 8, dim, dtype, 16, 1 << 20, 1 << 16, max_q,
                                      max_kv, window=window)
            assert sffn.paged_attn_mx4_workspace_bytes(b) <= (256 << 20) + 1024
            b.T -= max_q - 1      # both kernels may have to run
            assert sffn.paged_attn_mx4_workspace_bytes(b) <= 2 * (256 << 20) + 2048


# ---------------------------------------------------------------- the binding
def cache_of(sffn, n_pages=4, page=16, heads=2, dim=64, **kw):  # noqa: F811
    t = dict(k_codes=gpu(n_pages, page, heads, dim // 2, dtype=torch.uint8),
             k_scales=gpu(n_pages, page, heads, -(-dim // 32), dtype=torch.uint8))
    t.update(v_codes=t["k_codes"], v_scales=t["k_scales"])
    t.update(kw)
    return sffn.Mx4Cache(n_pages, page, heads, dim, **t)


def test_struct_layout(sffn):  # noqa: F811
    assert ctypes.sizeof(sffn.Mx4Rows) == 64


def test_tensors_of_a_cache(sffn):  # noqa: F811
    c = cache_of(sffn)
    assert c._k.token == 64 and c._k.scale_head == 2 and c.k_codes is not None
    # one byte of scales a row: its dimension has no stride
    cache_of(sffn, dim=24, k_scales=OnGpu(torch.zeros((4, 16, 2, 7), dtype=torch.uint8)[..., ::7]))
    u8 = torch.uint8
    for bad in (dict(k_codes=gpu(4, 16, 2, 64, dtype=u8)), dict(v_scales=gpu(4, 16, 2, 1, dtype=u8)),
                dict(v_codes=gpu(4, 16, 3, 32, dtype=u8)), dict(k_scales=gpu(5, 16, 2, 2, dtype=u8))):
        with pytest.raises(ValueError, match="must be"):
            cache_of(sffn, **bad)
    with pytest.raises(TypeError, match="uint8"):
        cache_of(sffn, k_codes=gpu(4, 16, 2, 32, dtype=torch.int8))
    with pytest.raises(ValueError, match="contiguous"):
        cache_of(sffn, v_codes=OnGpu(torch.zeros((4, 16, 2, 64), dtype=u8)[..., ::2]))
    with pytest.raises(ValueError, match="together"):
        cache_of(sffn, v_codes=None)
    with pytest.raises(ValueError, match="multiple of 8"):
        cache_of(sffn, dim=20)
    with pytest.raises(ValueError, match="GPU"):
        cache_of(sffn, k_codes=torch.zeros((4, 16, 2, 32), dtype=u8))


def attention(sffn, **kw):  # noqa: F811
    """8 rows of 2 sequences, 4 heads on 2 of 64, 4 pages of 16, 5 columns of pages; refused by
    the library (the scale is NaN)."""
    b = sffn.make_paged_batch(8, 2, 4, 2, 64, torch.bfloat16, 16, 4, 5, 4, 64, scale=float("nan"))
    a = dict(q=gpu(8, 4, 64), cache=cache_of(sffn), q_start=gpu(3, dtype=torch.int32),
             kv_len=gpu(2, dtype=torch.int32), block_table=gpu(2, 5, dtype=torch.int32), out=gpu(8, 4, 64),
             workspace=gpu(1024, dtype=torch.uint8), lse=gpu(8, 4, dtype=torch.float32))
    a.update(kw)
    sffn.paged_attn_mx4_fwd(b, stream=_NoStream, **a)


def appended(sffn, **kw):  # noqa: F811
    h = sffn.make_heads(8, 4, 2, 64, torch.bfloat16, norm=True, eps=float("nan"))
    a = dict(q=gpu(8, 4, 64), k=gpu(8, 2, 64), v=gpu(8, 2, 64), q_weight=gpu(64), k_weight=gpu(64),
             table=None, positions=None, slots=gpu(8, dtype=torch.int32), q_out=gpu(8, 4, 64),
             cache=cache_of(sffn))
    a.update(kw)
    sffn.paged_kv_append_mx4(h, stream=_NoStream, **a)


def read_back(sffn, **kw):  # noqa: F811
    a = dict(cache=cache_of(sffn), slots=gpu(8, dtype=torch.int32), k_out=gpu(8, 2, 64), v_out=gpu(8, 2, 64))
    a.update(kw)
    a["cache"].page_size = 0          # what the library refuses
    sffn.paged_kv_read_mx4(stream=_NoStream, **a)


def test_binding_checks(sffn):  # noqa: F811
    for call in (attention, appended, read_back):
        with pytest.raises(sffn.SffnError, match="status -1"):
            call(sffn)
    for bad in (cache_of(sffn, n_pages=5), cache_of(sffn, page=8), cache_of(sffn, heads=4), cache_of(sffn, dim=128)):
        with pytest.raises(ValueError, match="paged_attn_mx4_fwd: the cache has"):
            attention(sffn, cache=bad)
    for bad in (cache_of(sffn, heads=4), cache_of(sffn, dim=128)):
        with pytest.raises(ValueError, match="paged_kv_append_mx4: the cache has"):
            appended(sffn, cache=bad)
        with pytest.raises(ValueError, match="k_out must be"):
            read_back(sffn, cache=bad)
    with pytest.raises(ValueError, match="v must be"):
        appended(sffn, v=gpu(8, 4, 64))
    with pytest.raises(ValueError, match="k_weight must have 64 elements"):
        appended(sffn, k_weight=gpu(2, 64))
    with pytest.raises(ValueError, match="slots must have 8 elements"):
        appended(sffn, slots=gpu(7, dtype=torch.int32))
    with pytest.raises(TypeError, match="slots must be"):
        read_back(sffn, slots=gpu(8, dtype=torch.int64))
    with pytest.raises(TypeError, match="v_out must be"):
        read_back(sffn, v_out=gpu(8, 2, 64, dtype=torch.float32))
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        read_back(sffn, k_out=gpu(8, 2, 64, dtype=torch.float16), v_out=None)
    with pytest.raises(ValueError, match="block_table must have 5 columns"):
        attention(sffn, block_table=gpu(2, 6, dtype=torch.int32))
    sffn.paged_kv_read_mx4(cache_of(sffn), None, None, None)     # nothing to read


def test_tensors_of_another_device(sffn, monkeypatch):  # noqa: F811
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)
    here = 0
    monkeypatch.setattr(OnGpu, "get_device", lambda self: here, raising=False)
    monkeypatch.setitem(globals(), "_NoStream", None)
    for call in (attention, appended, read_back):
        here = 0
        with pytest.raises(ValueError, match="on GPU 0, the current device is 1"):
            call(sffn)
        here = 1
        with pytest.raises(sffn.SffnError, match="status -1"):
            call(sffn)


def test_paged_attention_takes_one_form(sffn):  # noqa: F811
    with pytest.raises(ValueError, match="4-bit cache is given as mx4"):
        sffn.PagedAttention(1, 1, 2, 1, 64, torch.bfloat16, 16, 4, 4, 1, 64, k_cache=gpu(4, 16, 1, 64),
                            mx4=True, device="cpu")
    with pytest.raises(ValueError, match="PagedAttention: the cache has"):
        sffn.PagedAttention(1, 1, 4, 2, 64, torch.bfloat16, 16, 5, 4, 1, 64, mx4=cache_of(sffn), device="cpu")
