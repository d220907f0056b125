"""The decoder block of examples/ served with a 4-bit cache, against whole sequences over the
keys and values that such a cache holds."""
from __future__ import annotations

import pytest

from test_gpu_block import block  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lengths,chunk,tokens", [((150, 37, 90), 48, 6), ((1,), 1, 3), ((64, 65), 200, 2)])
def test_serving_matches_whole_sequences(block, lengths, chunk, tokens):  # noqa: F811
    # the roundings of the block over a bf16 cache, without those of k and v (what is held is
    # the same on both sides, but for codes of keys whose projections round apart in bf16)
    assert block.serve(lengths, chunk, tokens, mx4=True) < 10 * 2.0 ** -9
