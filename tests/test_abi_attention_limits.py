"""Sizes at and beyond what the attention side's launches take, on the host: refused
before anything is launched, and accepted up to the limit.  An accepted size shows as the
complaint about a missing buffer that is looked at next, so nothing is launched here."""
from __future__ import annotations

import pytest

from test_abi_attention import (ARG, UNSUPPORTED, append, attn, batch, heads, norm_rope,  # noqa: F401
                                norm_rope_bwd, sffn)

NONE = (None, 512, 64)


@pytest.mark.parametrize("kw,status", [
    # single tokens, head_dim 128: workgroups of four waves, 2^32 threads are too many
    (dict(n_seqs=1 << 20, n_q_heads=16, n_kv_heads=16, head_dim=128), UNSUPPORTED),
    (dict(n_seqs=(1 << 20) - 1, n_q_heads=16, n_kv_heads=16, head_dim=128), ARG),
    # head_dim 64: eight waves
    (dict(n_seqs=1 << 20, n_q_heads=8, n_kv_heads=8), UNSUPPORTED),
    (dict(n_seqs=1 << 20, n_q_heads=7, n_kv_heads=7), ARG),
    # products of tiles and key heads beyond 32 bits
    (dict(n_seqs=1 << 20, n_q_heads=2048, n_kv_heads=2048), UNSUPPORTED),
    (dict(n_seqs=1 << 20, n_q_heads=4096, n_kv_heads=4096), UNSUPPORTED),
    (dict(n_seqs=1 << 20, n_q_heads=4096, n_kv_heads=4096, max_kv=0), UNSUPPORTED),
    # chunks among many sequences: tiles of many rows, and items numbered on the device
    (dict(T=1 << 18, max_q=1000, n_seqs=1 << 18, n_q_heads=4096, n_kv_heads=4096), UNSUPPORTED),
    (dict(T=5000, max_q=1000, n_seqs=1 << 20, n_q_heads=4096, n_kv_heads=4096, max_kv=64), UNSUPPORTED),
    (dict(T=5000, max_q=1000, n_seqs=1 << 12, n_q_heads=64, n_kv_heads=8), ARG),
    # nothing but chunks: T = n_seqs * max_q
    (dict(T=1 << 18, max_q=1 << 6, n_seqs=1 << 12, n_q_heads=4096, n_kv_heads=1), ARG),
    (dict(T=1 << 18, max_q=65, n_seqs=1 << 18, n_q_heads=4096, n_kv_heads=4096, max_kv=0), UNSUPPORTED),
])
def test_grids_of_the_attention(sffn, kw, status):  # noqa: F811
    b = batch(sffn, **kw)
    assert attn(sffn, b, q=NONE) == status
    if status != ARG:
        assert sffn._lib.paged_attn_workspace_bytes(b) == 0


def test_grids_of_the_heads(sffn):  # noqa: F811
    """64 threads a token in the forward and the append; the backward walks over tokens."""
    for T, status in (((1 << 26) - 4, ARG), ((1 << 26) - 3, UNSUPPORTED), (1 << 26, UNSUPPORTED),
                      ((1 << 31) - 1, UNSUPPORTED)):
        h = heads(sffn, T=T)
        assert norm_rope(sffn, h, q=NONE) == status and append(sffn, h, q=NONE) == status
    for T, status in ((1 << 26, ARG), (1 << 30, ARG), ((1 << 30) + 1, UNSUPPORTED),
                      ((1 << 31) - 1, UNSUPPORTED)):
        h = heads(sffn, T=T)
        assert norm_rope_bwd(sffn, h, q=NONE) == status
        assert (sffn._lib.qk_norm_rope_bwd_workspace_bytes(h) > 0) == (status == ARG)


def test_rows_of_a_cache_fit_a_slot(sffn):  # noqa: F811
    h = heads(sffn)
    assert append(sffn, h, q=NONE, n_pages=1 << 27, page=16) == ARG
    assert append(sffn, h, q=NONE, n_pages=(1 << 27) + 1, page=16) == UNSUPPORTED
    assert append(sffn, h, q=NONE, n_pages=(1 << 31) - 1, page=(1 << 31) - 1) == UNSUPPORTED


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("max_q", [1, 8, 16, 500])
@pytest.mark.parametrize("window", [0, 5000])
def test_workspace_under_the_limits_of_a_model(sffn, dtype, dim, max_q, window):  # noqa: F811
    """max_kv is an upper bound and usually the model's limit: the partial results of single
    tokens, drafts and chunks stay within 256 MiB (and its rounding) for every batch."""
    import torch
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    for n_seqs in (1, 32, 64, 256, 512, 1024, 10000):
        for max_kv in (4096, 32768, 131072, 1 << 20):
            b = sffn.make_paged_batch(n_seqs * max_q, n_seqs, 32, 8, dim, dt, 16, 1 << 20, 1 << 16, max_q,
                                      max_kv, window=window)
            need = sffn.paged_attn_workspace_bytes(b)
            assert need <= (256 << 20) + 1024, (n_seqs, max_kv, need)
            # one sequence less than full: both kernels may have to run
            b.T -= max_q - 1
            assert sffn.paged_attn_workspace_bytes(b) <= 2 * (256 << 20) + 2048


def test_workspace_holds_the_rows_that_exist(sffn):  # noqa: F811
    """Single tokens of 4 heads a key head need 4 rows of partial results a split, not 32."""
    import torch
    b = sffn.make_paged_batch(32, 32, 32, 8, 128, torch.bfloat16, 16, 1 << 20, 1 << 16, 1, 4096)
    one = 32 * 8 * 4 * (128 + 2) * 4     # 32 sequences, 8 key heads, output, maximum and sum
    need = sffn.paged_attn_workspace_bytes(b)
    assert need % one <= 512 and 2 <= need // one <= 8, need / one
