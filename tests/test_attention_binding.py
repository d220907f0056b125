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


def rotated(sffn, name="qk_norm_rope", **kw):  # noqa: F811
    """The heads of q and k (forward, backward or append), 8 tokens, 4 heads on 2 of 64."""
    h = sffn.make_heads(8, 4, 2, 64, torch.bfloat16, norm=True, eps=float("nan"))
    q, k, w = gpu(8, 4, 64), gpu(8, 2, 64), gpu(64)
    a = dict(q_weight=w, k_weight=w)
    a.update(kw)
    head = [h, q, k] + ([k] if name == "paged_kv_append" else [])
    head += [a.pop("q_weight"), a.pop("k_weight"), None, None]
    if name == "qk_norm_rope":
        sffn.qk_norm_rope(*head, q, k, stream=_NoStream)
    elif name == "paged_kv_append":
        sffn.paged_kv_append(*head, gpu(8, dtype=torch.int32), q, gpu(4, 16, 2, 64),
                             gpu(4, 16, 2, 64), stream=_NoStream)
    else:
        g = gpu(64, dtype=torch.float32)
        sffn.qk_norm_rope_bwd(*head, q, k, q, k, a.get("gq_weight", g), a.get("gk_weight", g),
                              gpu(1 << 16, dtype=torch.uint8), stream=_NoStream)


def test_norm_weights_are_one_row(sffn):  # noqa: F811
    """Weights of every head would be taken for those of the first."""
    for name in ("qk_norm_rope", "paged_kv_append", "qk_norm_rope_bwd"):
        accepted(sffn, rotated, name=name)
        accepted(sffn, rotated, name=name, q_weight=gpu(1, 64), k_weight=None)
        for bad in (gpu(4, 64), gpu(128), gpu(60)):
            with pytest.raises(ValueError, match="q_weight must have 64 elements"):
                rotated(sffn, name=name, q_weight=bad)
            with pytest.raises(ValueError, match="k_weight must have 64 elements"):
                rotated(sffn, name=name, k_weight=bad)
    with pytest.raises(ValueError, match="gq_weight must have 64 elements"):
        rotated(sffn, "qk_norm_rope_bwd", gq_weight=gpu(4, 64, dtype=torch.float32))
    with pytest.raises(ValueError, match="gk_weight must have 64 elements"):
        rotated(sffn, "qk_norm_rope_bwd", gk_weight=gpu(2, 64, dtype=torch.float32))


def test_tensors_of_another_device(sffn, monkeypatch):  # noqa: F811
    """Without a stream the current device's is used: tensors of another are refused."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)
    here = 0
    monkeypatch.setattr(OnGpu, "get_device", lambda self: here, raising=False)
    for call in (attention, *(lambda m, n=n: rotated(m, n) for n in
                              ("qk_norm_rope", "paged_kv_append", "qk_norm_rope_bwd"))):
        monkeypatch.setitem(globals(), "_NoStream", None)   # the current stream
        here = 0
        with pytest.raises(ValueError, match="on GPU 0, the current device is 1"):
            call(sffn)
        here = 1
        accepted(sffn, call)


def test_slots_of_tokens_outside_the_table(sffn):  # noqa: F811
    """Padding tokens get no slot, not the last page's."""
    bt = torch.tensor([[4, 2, 7], [1, 0, -1]], dtype=torch.int32)
    seq = torch.tensor([0, 0, 0, 0, 0, 1, 1])
    pos = torch.tensor([-1, -15, 14, 15, 1 << 30, 3, 11])
    assert sffn.paged_slots(bt, seq, pos, 5).tolist() == [-1, -1, 39, -1, -1, 8, -1]
    assert sffn.paged_slots(bt, seq.int(), pos.int(), 5).dtype is torch.int32
