"""The example of adapters trained from preference pairs: the operators in one training and serving loop."""

import math
import os
import sys

import pytest

from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_preference_adapters():
    require_gpu()
    import preference_adapters

    losses, batch, alone = preference_adapters.run(steps=40, say=say)
    # L2 = 0: policy and reference rows have the same logits, every h_p is 0 up to the order of one row's sums
    assert abs(losses[0] - math.log(2)) < 1e-4
    assert sum(losses[-5:]) / 5 < 0.5 * losses[0]
    # a user's tokens are 1 in 6 of the vocabulary
    assert sum(batch) / len(batch) > 0.5
    assert sum(alone) / len(alone) > 0.5
