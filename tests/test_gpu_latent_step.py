"""The example of steps on a paged latent cache: forks share the prompt's blocks, every emitted token is the one that the cache
names, and the reference counts are those of the rows.

Why no other token can win: normalised names and values are +-1 in 128 places each (times 1.1 for decoded tokens), so a right
key scores 128 a head, a wrong one 1.1 times a sum of 128 random signs at most: below 90 for all pairs of the 41 names in both
layers with probability 1 - 1e-9 (Hoeffding), and the rotated part adds 0.1 at most. sm_scale 0.25 puts e^-9 between them, and
the answer's logit, 128 a layer, is then off by less than a hundredth of what lies between the values' products."""

import os
import sys

import pytest

from gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,seed", [(1, 0), (4, 1), (9, 2)])
def test_latent_step(B, seed):
    need_gpu()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import latent_step

    emitted, right, mean, target = latent_step.run(steps=12, B=B, seed=seed)
    assert emitted == right
    assert mean > 1.5  # several tokens a step are accepted
    rows = target.table.cpu()
    counts = [0] * target.refs.numel()
    for i in rows[rows >= 0].tolist():
        counts[i] += 1
    assert target.refs.tolist() == counts
    shared = latent_step.TOKENS // latent_step.BLOCK  # the prompt's full blocks are held by all
    assert all(rows[b, :shared].tolist() == rows[0, :shared].tolist() for b in range(B))
    assert len({int(rows[b, shared]) for b in range(B)}) == B
