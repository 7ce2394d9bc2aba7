"""Attention over the paged latent cache in every kernel that the dispatch knows, each reached on purpose: signs and sizes of the
scale, references that move, what some rows do not see, and the same bits in every call."""

import math

import pytest
import torch

import latent_plain as plain
from gpu_helpers import need_gpu
from latent_dispatch import item_rows
from test_gpu_latent import attend, close, queries, tree_mask

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
SCALE = 192 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


# heads of 9 step tokens, latent dimensions, rows of an item
KERNELS = [(1, 128, 16), (3, 256, 32), (5, 384, 48), (5, 512, 48), (7, 256, 64), (16, 384, 64), (16, 512, 64),
           (15, 128, 128), (15, 256, 128), (24, 384, 128), (24, 512, 128), (40, 512, 128)]


@pytest.mark.parametrize("heads,C,rows", KERNELS)
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("scale", [-SCALE, 0.0, 1e-30, 3.0, -3.0])
def test_scales(heads, C, rows, dt, scale):
    c = plain.Cache([70, 200], [9, 9], C, 64, 32, dt, seed=1).fill()
    assert item_rows(c, heads, 9) == rows
    q = queries(c, heads, 4, 0.2)
    close(attend(c, q.cuda(), scale=scale)["out"], *plain.attention(c, q, scale), scale)


@pytest.mark.parametrize("heads,C,rows", KERNELS)
@pytest.mark.parametrize("dt", [BF, HF])
def test_scores_that_rise(heads, C, rows, dt):
    """Every tile's scores pass the last one's by far more than 2^8 and 2^15, or stay far below them; or rise by less, so that some
    tiles move references and some do not. 40 sequences, most of them whole items of several tiles."""
    B = 40
    c = plain.Cache([900] * 2 + [300] * (B - 2), [1, 9] + [1] * (B - 2), C, 16, 64, dt, seed=2).fill(0.05)
    assert item_rows(c, heads, 9) == rows
    q = queries(c, heads, 5, 0.05)
    q[..., 0] = 4.0
    for b in range(B):
        for t in range(c.ctx[b]):
            blk, s = c.slot(b, t)
            c.pool[blk, s, 0] = (t // 64) * (30.0, -30.0, 2.0)[b % 3]
    close(attend(c, q.cuda(), scale=1.0)["out"], *plain.attention(c, q, 1.0))


@pytest.mark.parametrize("heads,C,rows", KERNELS)
@pytest.mark.parametrize("dt", [BF, HF])
def test_what_no_row_sees(heads, C, rows, dt):
    """Infinities and NaN in the first values, the last ones or all over an entry of the step that only some rows see."""
    n, bad = 9, 4
    mask = tree_mask(8, 2, n)
    mask[:, :, bad] = 0
    mask[0, bad:, bad] = 1  # the second sequence's rows never see it
    mask[1, 1] = 0  # a row without anything
    for dims in (slice(0, 2), slice(C - 2, C), slice(3, C, 7)):
        c = plain.Cache([130, 0], [n, n], C, 32, 32, dt, seed=6).fill()
        clean = plain.Cache([130, 0], [n, n], C, 32, 32, dt, seed=6).fill()
        assert item_rows(c, heads, n) == rows
        q = queries(c, heads, 7)
        for b, x in ((0, math.nan), (1, math.inf)):
            blk, s = c.slot(b, c.ctx[b] + bad)
            c.pool[blk, s, dims] = x
        r = attend(c, q.cuda(), mask=mask)
        assert r["row_status"].tolist() == [0, 0]
        sees = mask.clone()
        sees[0, bad:] = 0
        want, tol = plain.attention(clean, q, SCALE, sees)
        rows_ = torch.ones(2 * n, dtype=torch.bool)
        rows_[bad:n] = False
        close(r["out"][rows_.cuda()], want[rows_], tol[rows_])
        assert bool(torch.isnan(r["out"][bad:n]).all()) and bool((r["out"][n + 1] == 0).all())
        r = attend(c, q.cuda())  # under the causal mask, rows before the entry
        want, tol = plain.attention(clean, q, SCALE)
        for b in range(2):
            close(r["out"][b * n: b * n + bad], want[b * n: b * n + bad], tol[b * n: b * n + bad])
        assert bool(torch.isnan(r["out"][bad:n]).all())


@pytest.mark.parametrize("heads,C,rows", KERNELS)
def test_the_same_bits(heads, C, rows):
    c = plain.Cache([700, 20, 1300] * 9, [9, 4, 1] * 9, C, 64, 64, BF, seed=30).fill()
    assert item_rows(c, heads, 9) == rows
    q, args = queries(c, heads, 31).cuda(), c.to("cuda")
    first = attend(c, q, args)["out"]
    for _ in range(8):
        assert torch.equal(attend(c, q, args)["out"], first)
