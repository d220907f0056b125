"""Batches that the header says are taken, at the limits of a grid (no GPU needed)."""
from __future__ import annotations

import pytest

from test_abi_attention import ARG, UNSUPPORTED, batch, sffn  # noqa: F401
from test_abi_mx4 import NONE, attn


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("head_dim", [64, 128, 136, 256])
@pytest.mark.parametrize("g", [1, 16, 17, 32])
@pytest.mark.parametrize("max_kv", [100, 1000, 1280, 1281, 1600])
def test_many_sequences_of_few_rows(sffn, dtype, head_dim, g, max_kv):  # noqa: F811
    """n_seqs times n_kv_heads below 2^23, up to 32 rows a sequence: what is refused is a missing
    buffer."""
    for n_seqs, hkv in (((1 << 20) - 1, 8), (1 << 20, 7), (1 << 13, 1023)):
        kw = dict(n_seqs=n_seqs, n_q_heads=min(g, 4096 // hkv) * hkv, n_kv_heads=hkv, head_dim=head_dim, dtype=dtype,
                  max_q=1, max_kv=max_kv)
        assert attn(sffn, batch(sffn, **kw), q=NONE) == ARG


def test_more_may_be_refused(sffn):  # noqa: F811
    kw = dict(n_seqs=1 << 20, n_q_heads=256, n_kv_heads=16, head_dim=256, max_q=1, max_kv=1000)
    assert attn(sffn, batch(sffn, **kw), q=NONE) == UNSUPPORTED
