"""Attention up to the stated limit of sums: values whose magnitudes, summed over the keys that
a row sees, stay below 2^119 give finite results, over both caches."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import test_gpu_attention as P
import test_gpu_mx4 as M
from test_gpu_attention import E, U

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("q_lens,kv_lens", [([1], [2]), ([1, 4], [700, 33]), ([1], [9000]), ([150], [900]),
                                            ([150], [150]), ([100], [3000])])
def test_sums_below_the_limit(q_lens, kv_lens, D, dtype):
    """All keys have the same value, so that it is the result of every row.  Scores rise by 2^7.9
    after the first keys: the weights are relative to an older maximum, as large as they get.
    The result errs by the roundings of the weights and sums (twice, numerator and denominator)
    and its own."""
    c = P._attention_case(q_lens, kv_lens, 4, 2, D, 16, dtype, seed=51)
    n = max(kv_lens)
    e = math.floor(119 - math.log2(1.5 * n))
    c["q"][:] = 0.0
    c["q"][..., 0] = 1.0
    value = 1.5 * 2.0 ** e * torch.where(torch.arange(D) % 3 == 0, -1.0, 1.0).double()
    for b, length in enumerate(kv_lens):
        for j in range(length):
            at = int(c["bt"][b, j // 16]), j % 16
            c["k"][at] = 0.0
            c["k"][at][:, 0] = 0.0 if j < 256 else 4.0
            c["v"][at] = value.to(c["v"])
    scale = 7.9 / (4.0 * math.log2(math.e))
    out, _ = P._run(c, sm_scale=scale)
    rel = 2 * (n + 64) * U + (2 * E if dtype == "bf16" else 0.0) + (E if dtype == "bf16" else U)
    want = value.numpy()
    assert (np.abs(out.double().cpu().numpy() - want) <= rel * np.abs(want)).all()
    M._quantised(c)
    out, _ = M._run(c, sm_scale=scale)
    assert (np.abs(out.double().cpu().numpy() - want) <= rel * np.abs(want)).all()
