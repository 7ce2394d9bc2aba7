"""Attention over the 8-bit paged cache: scales below and at zero, and more sequences than a thread block has threads, so that
its run is searched in several rounds. Tolerances are those of kv8_rows."""

import random

import pytest
import torch

import kv8_plain as plain
import kv8_rows
from gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def run(c, q, scale, most, tree=None):
    import speculative_decoding_verification_29_gb300 as sv

    r = sv.spec_kv8_attention(q.cuda(), *c.to("cuda"), c.cu.cuda(), max_tokens=most, sm_scale=scale,
                              tree_mask=None if tree is None else tree.cuda())
    torch.cuda.synchronize()
    kv8_rows.check(c, q, r["out"].cpu().double(), r["row_status"].tolist(), scale, most, tree)


@pytest.mark.parametrize("scale", [-0.1, -2.0, 0.0, -0.0, 1e-30, 1e-42])
@pytest.mark.parametrize("ctx,new,Hq,H,D,dt,tree", [
    ([200, 5], [1, 1], 8, 2, 128, BF, False),
    ([300, 70], [9, 4], 8, 2, 64, HF, False),
    ([130, 0], [16, 16], 8, 2, 128, BF, True),
    ([150, 20], [40, 33], 4, 2, 128, HF, True),
    ([90, 300], [200, 130], 4, 2, 128, BF, False),
])
def test_scales_below_and_at_zero(ctx, new, Hq, H, D, dt, tree, scale):
    c = plain.Cache(ctx, new, H, D, 32, seed=Hq).fill(spread=0.5)
    mask = None
    if tree:
        mask = plain.tree_mask(random.Random(1), len(ctx), max(new))[0]
        mask[0, 3] = 0  # with no context (below), a row that sees nothing
    q = torch.randn(sum(new), Hq, D, generator=torch.Generator().manual_seed(3)).to(dt)
    run(c, q, scale, max(new), mask)


MANY = [
    # sequences, step tokens of one, the most, query heads of a KV head, D, block, leading sequences without tokens
    (900, [0, 1], 1, 4, 64, 16, 0),  # 16 rows, 224 threads a block
    (1500, [0, 1, 2, 16], 16, 4, 64, 16, 0),  # 64 rows, 640 threads
    (1100, [0, 0, 1, 20], 20, 4, 64, 32, 0),  # 80 rows, 512 threads
    (600, [0, 1, 2], 300, 1, 128, 16, 0),  # 256 rows and two row tiles a sequence
    (1000, [0, 1, 3], 4, 4, 64, 16, 950),  # nothing in the first rounds
    (1300, [0], 300, 1, 64, 16, 1299),  # one sequence behind all the others
]


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("B,some,most,group,D,bs,empty", MANY)
def test_more_sequences_than_threads(B, some, most, group, D, bs, empty, dt):
    rng = random.Random(B)
    new = [0 if b < empty else rng.choice(some) for b in range(B)]
    new[B - 1] = most
    new[B // 2] = most if not empty else 0
    ctx = [rng.choice([0, rng.randint(0, 20), rng.randint(0, 60)]) for _ in range(B)]
    for b in rng.sample(range(B), 12):
        ctx[b] = rng.randint(100, 700)
    ctx[B - 1] = 900
    c = plain.Cache(ctx, new, 1, D, bs, seed=most).fill(spread=0.5)
    q = torch.randn(sum(new), group, D, generator=torch.Generator().manual_seed(6)).to(dt)
    run(c, q, D ** -0.5, most)
