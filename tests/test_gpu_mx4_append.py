"""Appends into the 4-bit cache whose keys lie on borders between two codes, or are zero: the bytes
are those of 64-bit arithmetic."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from helpers import to_f64
from oracle import attention as A
from oracle import mx4
from test_gpu_attention import DT, _randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("zeros", [0.0, 0.01, 1.0])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("T,D,rot,adjacent", [
    (300, 128, 64, False), (300, 128, 32, True), (2100, 128, 96, False), (70, 80, 40, False), (70, 80, 20, True),
    (40, 256, 36, False), (40, 24, 12, True), (65, 64, 64, False)])
def test_rotated_in_part(T, D, rot, adjacent, norm, zeros, dtype):
    """What is not rotated, without a norm, is the input itself: in bf16 often right on a border."""
    from activation_sparse_feed_amd import sffn
    rng = np.random.default_rng(T + D)
    hkv, page = 3, 16
    qkv = _randn(rng, (T, 2 + 2 * hkv, D), dtype)
    qkv[torch.from_numpy(rng.random(tuple(qkv.shape)) < zeros).cuda()] = 0.0
    qkv *= torch.from_numpy(rng.choice([-1.0, 1.0], qkv.shape).astype(np.float32)).cuda().to(qkv.dtype)   # and -0
    q, k, v = qkv[:, :2], qkv[:, 2:2 + hkv], qkv[:, 2 + hkv:]
    pos = rng.integers(0, 4096, T).astype(np.int32)
    tab = sffn.rotary_table(4096, rot)
    n_pages = -(-T // page)
    cache = sffn.Mx4Cache(n_pages, page, hkv, D)
    h = sffn.make_heads(T, 2, hkv, D, DT[dtype], rot, 4096, norm, 1e-5, adjacent)
    slots = rng.permutation(n_pages * page)[:T].astype(np.int32)
    qo = torch.empty((T, 2, D), dtype=DT[dtype], device="cuda")
    sffn.paged_kv_append_mx4(h, q, k, v, None, None, tab, torch.from_numpy(pos).cuda(),
                             torch.from_numpy(slots).cuda(), qo, cache)
    rows = A.norm_rope(to_f64(k), None, to_f64(tab), pos, rot, adjacent, norm, float(np.float32(1e-5)))
    for n, want in (("k", rows.astype(np.float32)), ("v", to_f64(v))):
        codes, scales = mx4.encode(want)
        have = [getattr(cache, f"{n}_{x}").cpu().numpy()[slots // page, slots % page] for x in ("codes", "scales")]
        assert np.array_equal(have[1], scales) and np.array_equal(have[0], codes), n
