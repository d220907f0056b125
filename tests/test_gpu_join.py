"""The join of split key ranges where it loads parts early (many splits, few workgroups, few bytes)
and where it does not, on both sides of each border, over both caches."""
from __future__ import annotations

import numpy as np
import pytest

import test_gpu_attention as P
import test_gpu_mx4 as M
from test_gpu_mx4_values import check_values

pytestmark = pytest.mark.gpu

SPLITS = [
    # kv_lens, max_kv: bf16 ranges of width 128 are cut into 256 keys or more
    ([300, 1], 300), ([700, 40, 1], 700), ([1500, 2, 640], 1500), ([4096, 3, 900], 4096),   # 16 splits
    ([4097, 257, 0], 4097), ([5500, 100], 5500), ([20000, 33], 20000),                      # 17, 22, 64
    ([900, 40, 3], 200000),                 # hardly any part is written, none of the third
    ([5000] + [int(n) for n in np.linspace(1, 5000, 36)], 5000),                            # more workgroups
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kv_lens,max_kv", SPLITS)
def test_joined_rows(kv_lens, max_kv, dtype):
    q_lens = [min(n, 1 + 2 * (i % 2)) for i, n in enumerate(kv_lens)]
    args = (q_lens, kv_lens, 8, 2, 128, 16, dtype)
    # the table has columns for max_kv
    def wide(c):
        more = -(-max_kv // 16) - c["bt"].shape[1]
        if more > 0:
            c["bt"] = np.concatenate([c["bt"], np.full((len(kv_lens), more), -1, np.int32)], 1)
        return c

    c = wide(P._attention_case(*args, seed=41))
    out, lse = P._run(c, max_kv=max_kv)
    P._check_attention(c, out, lse)
    c = wide(M._case(*args, seed=41))
    out, lse = M._run(c, max_kv=max_kv)
    check_values(c, out, lse)
