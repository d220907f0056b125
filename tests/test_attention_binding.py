"""The binding's checks of the attention side's arguments (no GPU needed): CPU tensors with a
GPU's flag, in calls that the library itself refuses (a scale or an eps that is NaN), so
that nothing is launched whatever the binding accepts."""
from __future__ import annotations

import pytest
import torch

from test_abi_attention import sffn  # noqa: F401


class OnGpu:
    """A CPU tensor with a GPU's flag."""

    def __init__(self, t):
        self.t, self.is_cuda = t, True

    def __getattr__(self, name):
        return getattr(self.t, name)


def gpu(*shape, dtype=torch.bfloat16):
    return OnGpu(torch.zeros(shape, dtype=dtype))


def attention(sffn, **kw):  # noqa: F811
    """8 rows of 2 sequences, 4 heads on 2 of 64, 4 pages of 16, 5 columns of pages."""
    b = sffn.make_paged_batch(8, 2, 4, 2, 64, torch.bfloat16, 16, 4, 5, 4, 64, scale=float("nan"))
    a = dict(q=gpu(8, 4, 64), k_cache=gpu(4, 16, 2, 64), v_cache=gpu(4, 16, 2, 64),
             q_start=gpu(3, dtype=torch.int32), kv_len=gpu(2, dtype=torch.int32),
             block_table=gpu(2, 5, dtype=torch.int32), out=gpu(8, 4, 64),
             workspace=gpu(1024, dtype=torch.uint8), lse=gpu(8, 4, dtype=torch.float32))
    a.update(kw)
    sffn.paged_attn_fwd(b, stream=_NoStream, **a)


class _NoStream:
    cuda_stream = 0


def accepted(sffn, call, **kw):  # noqa: F811
    with pytest.raises(sffn.SffnError, match="status -1"):
        call(sffn, **kw)


def test_columns_of_the_tables(sffn):  # noqa: F811
    accepted(sffn, attention)
    accepted(sffn, attention, lse=None)
    accepted(sffn, attention, block_table=gpu(3, 5, dtype=torch.int32))   # more rows
    accepted(sffn, attention, block_table=gpu(10, dtype=torch.int32))     # flat
    for cols in (6, 100, 10):
        with pytest.raises(ValueError, match="block_table must have 5 columns"):
            attention(sffn, block_table=gpu(2, cols, dtype=torch.int32))
    with pytest.raises(ValueError, match="block_table must have"):
        attention(sffn, block_table=gpu(1, 5, dtype=torch.int32))
    with pytest.raises(ValueError, match="lse must have 4 columns"):
        attention(sffn, lse=gpu(4, 8, dtype=torch.float32))
