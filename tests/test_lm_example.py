"""The example runs the operators together and its loss falls."""
from __future__ import annotations

import math

import pytest

pytestmark = pytest.mark.gpu


def test_head_learns_and_scores_alike():
    from examples.lm_head_step import train
    losses, found = train(steps=20, tokens=300, hidden=264, vocab=1003)
    # at first a little above ln(vocab), since the random head's logits spread
    assert abs(losses[0] - math.log(1003)) < 0.3
    assert losses[-1] < 0.7 * losses[0]
    # a token's loss alone and in a batch: the same products, cut differently along K
    assert found["single_token_difference"] < 1e-4
    # an e4m3 rounding is off by at most 2^-4 of a value, by less than half of that on average
    assert found["norm_8bit_relative_difference"] < 0.05
