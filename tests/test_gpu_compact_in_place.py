"""Compaction whose new lengths are written over the old ones or over the accepted lengths, in as many planes as give a
sequence several thread blocks: the same entries and lengths as with outputs of their own."""

import random

import pytest
import torch

import latent_plain as plain
from gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def sv():
    import speculative_decoding_verification_29_gb300 as m

    return m


def steps(B, D=12, N=40, ctx=60, seed=3):
    """Lengths, accepted lengths (one is none) and paths."""
    rng = random.Random(seed)
    acc = [rng.randint(1, D - 1) for _ in range(B)]
    acc[B // 2] = -1
    path = torch.full((B, D), -1, dtype=I32)
    for b, L in enumerate(acc):
        row = [0] + sorted(rng.sample(range(1, N), max(L, 0)))
        path[b, : len(row)] = torch.tensor(row, dtype=I32)
    lens = [rng.randint(0, ctx) for _ in range(B)]
    return torch.tensor(lens, dtype=I32), torch.tensor(acc, dtype=I32), path


def same_in_place(call, fresh, lens, acc, path):
    """call(caches, lengths, accepted, path, out): every choice of memory for new_len against outputs of their own."""
    want = fresh()
    w = call(want, lens.cuda(), acc.cuda(), path, None)
    for over in ("lengths", "accepted", "status over accepted"):
        caches, n, a = fresh(), lens.cuda(), acc.cuda()
        other = torch.empty_like(n)
        out = dict(new_len=n if over == "lengths" else a, row_status=other)
        if over == "status over accepted":
            out = dict(new_len=other, row_status=a)
        r = call(caches, n, a, path, out)
        assert torch.equal(r["new_len"], w["new_len"]) and torch.equal(r["row_status"], w["row_status"]), over
        for x, y in zip(caches, want):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), over


@pytest.mark.parametrize("planes", [1, 2, 32])
@pytest.mark.parametrize("chain", [False, True])
def test_latent(planes, chain):
    B, bs = 70, 16
    lens, acc, path = steps(B)
    c = plain.Cache(lens.tolist(), [40] * B, 512, 64, bs, torch.bfloat16, seed=5).fill()
    pool = torch.stack([c.pool.roll(i, 1) for i in range(planes)])
    t = c.table.cuda()

    def call(caches, n, a, p, out):
        return sv().spec_latent_compact(caches[0], t, n, a, None if chain else p.cuda(), out=out)

    same_in_place(call, lambda: [pool.cuda()], lens, acc, path)


@pytest.mark.parametrize("planes", [1, 24])
@pytest.mark.parametrize("chain", [False, True])
def test_kv8(planes, chain):
    B, bs, H, D = 70, 16, 8, 128
    lens, acc, path = steps(B, seed=6)
    M = 7
    g = torch.Generator().manual_seed(7)
    table = torch.randperm(B * M, generator=g).to(I32).view(B, M).cuda()
    codes = torch.randint(0, 127, (2, planes, B * M, H, bs, D), generator=g, dtype=torch.uint8)  # finite ones
    scales = torch.randint(120, 134, (2, planes, B * M, H), generator=g, dtype=torch.uint8)

    def call(caches, n, a, p, out):
        return sv().spec_kv8_compact(*caches, table, n, a, None if chain else p.cuda(), out=out)

    same_in_place(call, lambda: [codes[0].cuda(), codes[1].cuda(), scales[0].cuda(), scales[1].cuda()], lens, acc, path)


@pytest.mark.parametrize("planes,W", [(1, 8), (64, 1024), (64, 1001)])
@pytest.mark.parametrize("chain", [False, True])
def test_kv(planes, W, chain):
    B = 9
    lens, acc, path = steps(B, seed=8)
    kv = torch.randn(planes, B, 110, W, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16)

    def call(caches, n, a, p, out):
        return sv().spec_kv_compact(caches[0], n, a, None if chain else p.cuda(), out=out)

    same_in_place(call, lambda: [kv.cuda()], lens, acc, path)
