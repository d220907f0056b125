"""The decoder block of examples/: served in chunks and single tokens against whole
sequences, and the head norms trained through the library's backward."""
from __future__ import annotations

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(__file__), "..", "examples", "decoder_block.py")


@pytest.fixture(scope="module")
def block():
    spec = importlib.util.spec_from_file_location("decoder_block", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("lengths,chunk,tokens", [((150, 37, 90), 48, 6), ((1,), 1, 3), ((64, 65), 200, 2)])
def test_serving_matches_whole_sequences(block, lengths, chunk, tokens):
    # q, k, v, the attention's output, both residuals and the FFN's input and
    # output are rounded to bf16 (2^-9 on average half an ulp) in both, and here the
    # weights of the softmax, the rotated heads and the FFN's h besides: about
    # ten roundings of 2^-9 each, in quadrature with their propagation
    assert block.serve(lengths, chunk, tokens) < 10 * 2.0 ** -9


def test_training_reaches_the_teacher(block):
    first, last = block.train()
    assert last < 1e-2 * first
