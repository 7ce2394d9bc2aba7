"""Appending under token ranges that do not rise: every sequence whose own range is sound gets all of its tokens, no other
entry changes, and the others are reported."""

import random

import pytest
import torch

import kv8_plain as plain
from gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def sv():
    import speculative_decoding_verification_29_gb300 as m

    return m


LISTS = [
    ([0, 100, 50, 100], 16),  # the third sequence shares the first one's last tokens
    ([0, 96, 2, 40], 16),
    ([60, 0, 61, 0, 62], 16),
    ([0, 300, 0, 300, 0, 300, 20, 310], 32),  # four long ranges over each other
    ([5, 5, 200, 130, 130, 290, 1], 64),
]


def random_lists():
    rng = random.Random(3)
    for bs in (16, 32, 128):
        yield [rng.randint(0, 200) for _ in range(rng.randint(3, 40))], bs


@pytest.mark.parametrize("cu,bs", LISTS + list(random_lists()))
def test_append_where_ranges_fall(cu, bs):
    B, T = len(cu) - 1, max(cu)
    new = [max(0, hi - lo) for lo, hi in zip(cu, cu[1:])]
    rng = random.Random(len(cu))
    ctx = [rng.choice([0, rng.randint(0, 2 * bs)]) for _ in new]
    c = plain.Cache(ctx, new, 2, 64, bs, seed=B).fill(upto=ctx)
    c.cu = torch.tensor(cu, dtype=torch.int32)
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(T, 2, 64, generator=g) * 2 for _ in range(2))
    q = torch.randn(T, 1, 64, generator=g)
    want, _ = plain.append(c, k, v)
    freq = [10000.0 ** (-i / 32) for i in range(32)]
    turned = {}  # each token's query at its place in every sequence that has it
    for b, lo in enumerate(cu[:-1]):
        for t in range(lo, cu[b + 1]):
            turned.setdefault(t, []).append(plain.rotate(q[t].double(), ctx[b] + t - lo, freq, False))
    for repeat in range(3):
        args = c.to("cuda")
        r = sv().spec_kv8_append(k.cuda(), v.cuda(), *args, c.cu.cuda(), q=q.cuda())
        assert r["row_status"].tolist() == [64 if hi < lo else 0 for lo, hi in zip(cu, cu[1:])]
        for i in range(4):
            assert torch.equal(args[i].cpu(), want[i]), (repeat, i)
    out = sv().spec_kv8_append(k.cuda(), v.cuda(), *c.to("cuda"), c.cu.cuda(), inv_freq=freq, q=q.cuda())["q_out"].cpu().double()
    for t, places in turned.items():  # fp32's turn: 2^-22 of the pair's size, below 8
        assert min(float((out[t] - w).abs().max()) for w in places) <= 2.0 ** -18
