"""The tree verification steps of examples/tree_step.py: every emitted token is the one that the target's memory holds.

Why no other token can win: names are +-1 in 96 unrotated places, so a right key scores 96 (or 1.25 times that, for decoded
tokens), a wrong one 1.25 times a sum of 96 random signs at most: below 75 for all pairs of the 41 names, layers and heads
with probability 1 - 1e-5, and 0.4 at most comes from the rotated part. sm_scale 0.25 puts e^-5 between even the worst pair
and the right one in one head, and 16 heads of other random names are summed. The codes hold +-1 and +-1.25 exactly."""

import os
import sys

import pytest

from gpu_helpers import need_gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,seed", [(1, 0), (4, 1), (13, 2)])
def test_walks_the_permutation(B, seed):
    need_gpu()
    import tree_step

    emitted, right, mean = tree_step.run(steps=30, B=B, seed=seed)
    assert emitted == right
    assert mean > 1.5  # the drafters' right guesses were accepted
