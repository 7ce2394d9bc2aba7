"""Attention over the 8-bit paged cache: a row's accuracy is its own, whatever the other heads and step tokens ask with."""

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


def run(c, q, scale=None, tree=None):
    import speculative_decoding_verification_29_gb300 as sv

    most = max(c.new) if tree is None else tree.shape[1]
    scale = c.D ** -0.5 if scale is None else scale
    r = sv.spec_kv8_attention(q.cuda(), *c.to("cuda"), c.cu.cuda(), max_tokens=most, sm_scale=scale,
                              tree_mask=None if tree is None else tree.cuda())
    torch.cuda.synchronize()
    kv8_rows.check(c, q, r["out"].cpu().double(), r["row_status"].tolist(), scale, most, tree)


CASES = [
    # ctx, new, Hq, H, D, tree: 8, 16, 36, 48, 64, 72, 128 and more rows
    ([700], [1], 8, 1, 128, False),
    ([300, 40], [4, 2], 8, 2, 64, False),
    ([500, 129], [9, 9], 8, 2, 128, False),
    ([200], [12], 8, 2, 64, False),
    ([260], [16], 8, 2, 128, False),
    ([400, 3], [18, 7], 8, 2, 128, False),
    ([150], [61], 4, 2, 64, True),
    ([30, 200], [150, 90], 4, 2, 128, False),
    ([100, 90], [20, 20], 6, 2, 128, True),
    ([100, 90], [40, 40], 14, 2, 64, True),
]


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("ctx,new,Hq,H,D,tree", CASES)
def test_rows_far_apart(ctx, new, Hq, H, D, tree, dt):
    """Heads and tokens whose queries are up to 2^12 times others', both ways round."""
    c = plain.Cache(ctx, new, H, D, 32, seed=Hq + D).fill(spread=0.5)
    mask = plain.tree_mask(random.Random(1), len(ctx), max(new))[0] if tree else None
    for seed in (1, 2):
        g = torch.Generator().manual_seed(seed)
        far = torch.tensor([0.0, 0.0, -4.0, 8.0, 10.0, 12.0])[torch.randint(0, 6, (sum(new), Hq, 1), generator=g)]
        run(c, (torch.randn(sum(new), Hq, D, generator=g) * 2.0 ** far).to(dt), tree=mask)


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("new", [9, 20])
def test_rows_without_finite_elements(dt, new):
    """A row of zeros, and one of infinities and NaN, move no other row."""
    import speculative_decoding_verification_29_gb300 as sv

    c = plain.Cache([300, 140], [new, new], 2, 128, 32, seed=11).fill(spread=0.5)
    q = torch.randn(2 * new, 8, 128, generator=torch.Generator().manual_seed(4))
    q[::2] *= 2.0 ** 9
    q[1, 3] = 0.0
    run(c, q.to(dt))
    call = lambda: sv.spec_kv8_attention(q.to(dt).cuda(), *c.to("cuda"), c.cu.cuda(), max_tokens=new)["out"]  # noqa: E731
    want = call()
    q[4, 6] = torch.where(torch.arange(128) % 2 == 0, float("inf"), float("nan"))
    got = call()
    assert torch.isnan(got[4, 6]).all()
    got[4, 6] = want[4, 6]
    assert torch.equal(got, want)


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("ctx,new,Hq,H,D,tree", CASES)
def test_rows_alike(ctx, new, Hq, H, D, tree, dt):
    """Queries of one size, to the bounds of the kernel that takes them."""
    c = plain.Cache(ctx, new, H, D, 64, seed=Hq + D + 1).fill(spread=1.0)
    mask = plain.tree_mask(random.Random(2), len(ctx), max(new))[0] if tree else None
    run(c, (torch.randn(sum(new), Hq, D, generator=torch.Generator().manual_seed(3)) * 1.5).to(dt), tree=mask)
