"""Attention over the paged latent cache where an entry has one infinite element: rows whose score is then +infinity are NaN,
those whose score is -infinity are NaN in that dimension alone (none, where it is a shared one), whichever kernel runs, whether
the entry belongs to the context or to the step, and rows that do not see it are as without it."""

import math

import pytest
import torch

import latent_plain as plain
from gpu_helpers import need_gpu
from latent_dispatch import item_rows

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
SCALE = 192 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def sv():
    import speculative_decoding_verification_29_gb300 as m

    return m


class Without:
    """A cache without one of the context's entries."""

    def __init__(self, c, b, t):
        self.c, self.b, self.t = c, b, t
        self.ctx, self.new, self.C, self.R, self.dt = list(c.ctx), c.new, c.C, c.R, c.dt
        self.ctx[b] -= 1

    def entries(self, b):
        e = self.c.entries(b)
        return e if b != self.b else torch.cat((e[: self.t], e[self.t + 1:]))


def tree(B, n):
    m = torch.zeros(B, n, n, dtype=torch.uint8)
    for i in range(n):
        if i:
            m[:, i] = m[:, (i - 1) // 2]
        m[:, i, i] = 1
    return m


# heads, step tokens, C, R, rows of an item
SHAPES = [(1, 9, 512, 64, 16), (3, 9, 384, 48, 32), (5, 9, 256, 32, 48), (7, 9, 512, 64, 64), (16, 9, 512, 64, 64), (24, 9, 512, 64, 128),
          (24, 9, 384, 48, 128), (15, 9, 256, 32, 128), (15, 9, 128, 16, 128)]


@pytest.mark.parametrize("where", ["context", "edge", "step", "first step token"])
@pytest.mark.parametrize("heads,n,C,R,rows", SHAPES)
@pytest.mark.parametrize("dt,masked", [(BF, False), (HF, True)])
def test_one_infinite_element(heads, n, C, R, rows, dt, masked, where):
    ctx, at = [300, 150], dict(context=3, edge=298, step=304)
    mask = tree(2, n) if masked else None
    for dim in (5, C - 3, C + 7):  # the first half of the values, the second, a shared one
        c = plain.Cache(ctx, [n, n], C, R, 32, dt, seed=C + dim).fill()
        assert item_rows(c, heads, n) == rows
        t = at.get(where, 300)
        g = torch.Generator().manual_seed(dim)
        q = (torch.randn(2 * n, heads, C + R, generator=g) * 0.7).to(dt)
        sign = torch.where(torch.rand(2 * n, heads, generator=g) < 0.8, -1.0, 1.0)
        q[..., dim] = sign.to(dt)  # the score's sign
        if t < 300:
            want, tol = plain.attention(Without(c, 0, t), q, SCALE, mask)
            saw = torch.ones(n, dtype=torch.bool)
        else:
            see = (mask if masked else torch.ones(2, n, n, dtype=torch.uint8).tril()).clone()
            saw = see[0, :, t - 300].bool()
            see[0, :, t - 300] = 0
            want, tol = plain.attention(c, q, SCALE, see)
        blk, s = c.slot(0, t)
        c.pool[blk, s, dim] = math.inf
        p, table, length = c.to("cuda")
        r = sv().spec_latent_attention(q.cuda(), p, table, length, c.cu.cuda(), max_tokens=n, value_dim=C, sm_scale=SCALE,
                                       tree_mask=None if mask is None else mask.cuda())
        assert r["row_status"].tolist() == [0, 0]
        got = r["out"].double().cpu()
        for i in range(2 * n):
            for h in range(heads):
                x = got[i, h]
                if i < n and saw[i] and sign[i, h] > 0:
                    assert bool(torch.isnan(x).all()), (dim, i, h)
                    continue
                ok = (x - want[i, h]).abs() <= tol[i, h]
                if i < n and saw[i] and dim < C:
                    assert bool(torch.isnan(x[dim])), (dim, i, h)
                    ok[dim] = True
                assert bool(ok.all()), (dim, i, h, int((~ok).sum()))


@pytest.mark.parametrize("heads,rows", [(7, 32), (120, 128)])
def test_whole_items(heads, rows):
    """Items of one tile: results that no join touches. Every sequence's last step token is infinite somewhere."""
    B, n, C = 90, 3, 512
    c = plain.Cache([i % 40 for i in range(B)], [n] * B, C, 64, 16, BF, seed=70).fill()
    assert item_rows(c, heads, n) == rows
    q = (torch.randn(B * n, heads, C + 64, generator=torch.Generator().manual_seed(71)) * 0.7).to(BF)
    q[..., 400] = -1.0
    see = torch.ones(B, n, n, dtype=torch.uint8).tril()
    see[:, :, n - 1] = 0
    want, tol = plain.attention(c, q, SCALE, see)
    for b in range(B):
        blk, s = c.slot(b, c.ctx[b] + n - 1)
        c.pool[blk, s, 400] = math.inf
    r = sv().spec_latent_attention(q.cuda(), *c.to("cuda"), c.cu.cuda(), max_tokens=n, value_dim=C, sm_scale=SCALE)
    got = r["out"].double().cpu()
    d = (got - want).abs()
    ok = d <= tol
    last = torch.arange(B * n) % n == n - 1
    assert bool(torch.isnan(got[last][..., 400]).all())
    ok[last, :, 400] = True
    assert bool(ok.all())
