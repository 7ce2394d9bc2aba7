"""Attention over the 8-bit paged cache with block ids outside the pool: the rows that see an entry of such a block are NaN, and
all others are right, whichever kernel takes them and however their item's tiles lie."""

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


CASES = [
    # ctx, new, Hq, H, D, block, position of the bad block, tree
    (0, 256, 1, 1, 128, 16, 130, False),  # rows of one item that see nothing of the bad block's tile
    (0, 300, 1, 1, 64, 128, 200, False),
    (40, 400, 2, 1, 128, 32, 300, False),
    (60, 100, 1, 1, 128, 64, 140, False),
    (120, 70, 2, 2, 128, 16, 180, False),
    (100, 48, 1, 1, 128, 16, 130, False),
    (110, 20, 3, 1, 64, 16, 125, False),
    (100, 61, 2, 1, 128, 16, 150, True),
    (120, 61, 4, 1, 128, 16, 160, True),
    (50, 30, 2, 1, 64, 32, 70, True),
    (500, 9, 4, 1, 128, 64, 0, False),  # seen by all
    (500, 80, 4, 1, 128, 64, 300, False),
]


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("ctx,new,Hq,H,D,bs,at,tree", CASES)
def test_block_outside_the_pool(ctx, new, Hq, H, D, bs, at, tree, dt):
    import speculative_decoding_verification_29_gb300 as sv

    c = plain.Cache([ctx, 30], [new, 2], H, D, bs, seed=new).fill()
    q = torch.randn(new + 2, Hq, D, generator=torch.Generator().manual_seed(5)).to(dt)
    mask = plain.tree_mask(random.Random(3), 2, new)[0] if tree else None
    want, tol = kv8_rows.attention(c, q, D ** -0.5, new, mask)
    page = at // bs
    bad = torch.arange(page * bs, (page + 1) * bs)
    hit = [bool((bad < ctx).any()) or any((mask[0, i, j] if tree else j <= i) for j in (bad - ctx).tolist() if 0 <= j < new)
           for i in range(new)] + [False, False]
    args = c.to("cuda")
    for outside in (-1, c.num, 2 ** 31 - 1):
        args[4][0, page] = outside
        r = sv.spec_kv8_attention(q.cuda(), *args, c.cu.cuda(), max_tokens=new, tree_mask=None if mask is None else mask.cuda())
        got = r["out"].cpu().double()
        assert r["row_status"].tolist() == [64, 0]
        for t, h in enumerate(hit):
            if h:
                assert torch.isnan(got[t]).all(), t
            else:
                assert ((got[t] - want[t]).abs() <= tol[t]).all(), t
    assert any(hit) and (not all(hit[:-2]) or at < ctx)
