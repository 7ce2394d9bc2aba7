"""The pages of a paged cache on the GPU against a step-by-step form: cutting back, forking, ending, taking and copying
blocks; pools of several types; too few blocks, unsound requests, in place and captured."""

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


def world(rng, B, M, bs, spare, shared=0.3):
    """Rows of random lengths, some of which share another's first blocks."""
    length = [rng.choice([0, rng.randint(0, M * bs), bs * rng.randint(0, M)]) for _ in range(B)]
    held = [-(-x // bs) for x in length]
    total = max(1, sum(held) + spare)
    ids = rng.sample(range(total), total)
    rows = []
    for b, k in enumerate(held):
        row = [ids.pop() for _ in range(k)]
        if b and rng.random() < shared:
            n = rng.randint(0, min(k, held[b - 1]))
            row[:n] = rows[-1][:n]
        rows.append(row + [-1] * (M - k))
    refs = [0] * total
    for row in rows:
        for i in row:
            if i >= 0:
                refs[i] += 1
    return torch.tensor(rows, dtype=I32), torch.tensor(length, dtype=I32), torch.tensor(refs, dtype=I32)


def check(table, length, refs, bs, pools=(), planes=False, block=None, **ask):
    want = plain.pages(table, length, refs, bs, ask.get("keep_len"), ask.get("source"), ask.get("need"))
    rows, lens, counts, status, copies = want
    dev = {k: v.cuda() for k, v in ask.items()}
    t, r = table.cuda(), refs.cuda()
    pools = [p.cuda() for p in pools]
    after = [p.clone() for p in pools]
    for p in after:
        for src, dst in copies:
            if planes:
                p[:, dst] = p[:, src]
            else:
                p[dst] = p[src]
    out = sv().spec_pages_update(t, length.cuda(), r, pools, planes=planes, block=block or bs, **dev)
    assert out["row_status"].tolist() == status
    assert out["block_table"].tolist() == rows
    assert out["cache_len"].tolist() == lens
    assert r.tolist() == counts and out["refs"] is r
    assert (out["block_table"] is t) == ("source" not in ask)
    if "source" in ask:
        assert torch.equal(t.cpu(), table)
    for p, w in zip(pools, after):
        assert torch.equal(p, w)
    return out, copies


@pytest.mark.parametrize("seed", range(12))
@pytest.mark.parametrize("fork", [False, True])
def test_random_steps(seed, fork):
    rng = random.Random(100 + seed)
    B, M, bs = rng.choice([1, 3, 17, 70]), rng.choice([1, 6, 40]), rng.choice([1, 4, 16])
    table, length, refs = world(rng, B, M, bs, rng.choice([0, 2, 5 * B]))
    source = [rng.randrange(B) for _ in range(B)] if fork else list(range(B))
    ask = dict(keep_len=torch.tensor([rng.choice([0, int(length[s]), rng.randint(0, int(length[s]))]) for s in source], dtype=I32),
               need=torch.tensor([rng.choice([0, 1, rng.randint(0, 2 * bs), M * bs]) for _ in range(B)], dtype=I32))
    if fork:
        ask["source"] = torch.tensor(source, dtype=I32)
    if seed % 4 == 1:
        del ask["keep_len"]
    if seed % 4 == 2:
        del ask["need"]
    check(table, length, refs, bs, **ask)


def test_many_sequences_and_blocks():
    rng = random.Random(7)
    table, length, refs = world(rng, 2100, 5, 8, 9000)
    need = torch.tensor([rng.randint(0, 20) for _ in range(2100)], dtype=I32)
    check(table, length, refs, 8, need=need)
    table, length, refs = world(rng, 3, 2500, 2, 6000)  # rows of several chunks
    check(table, length, refs, 2, source=torch.tensor([2, 2, 0], dtype=I32), need=torch.tensor([9, 2000, 1], dtype=I32))


@pytest.mark.parametrize("sixteen", [True, False])
def test_copies(sixteen):
    """Three forks of one sequence: all but the last copy its partly filled block, in every pool, or all where it is held elsewhere."""
    bs, nb = 16, 12
    g = torch.Generator().manual_seed(1)
    pools = [torch.randn(3, nb, bs, 144, generator=g).bfloat16(), torch.randint(0, 255, (3, nb, 2, bs, 64 if sixteen else 63),
                                                                             generator=g, dtype=torch.uint8),
             torch.randint(0, 255, (3, nb, 5), generator=g, dtype=torch.uint8)]
    table = torch.tensor([[4, 7, -1], [-1] * 3, [-1] * 3, [4, 7, -1]], dtype=I32)
    refs = torch.zeros(nb, dtype=I32)
    refs[4] = refs[7] = 2
    length = torch.tensor([20, 0, 0, 20], dtype=I32)
    source = torch.tensor([0, 0, 0, 3], dtype=I32)
    _, copies = check(table, length, refs, bs, pools, True, source=source, need=torch.tensor([3, 3, 3, 0], dtype=I32))
    assert copies == [(7, 0), (7, 1), (7, 2)]
    _, copies = check(table, length, refs, bs, pools, True, source=source, need=torch.tensor([3, 3, 3, 1], dtype=I32))
    assert copies == [(7, 0), (7, 1), (7, 2)]
    one = [p[1] for p in pools]
    _, copies = check(table, length, refs, bs, one, source=torch.tensor([0, 0, 0, 0], dtype=I32),
                      need=torch.tensor([3, 0, 20, 13], dtype=I32), keep_len=torch.tensor([20, 32 - 12, 20, 0], dtype=I32))
    assert copies == [(7, 0), (7, 1)]


def test_unsound_requests():
    table = torch.tensor([[0, 1], [2, -1], [3, 4], [5, 99]], dtype=I32)
    length = torch.tensor([20, 16, 32, 32], dtype=I32)
    refs = torch.tensor([1] * 6 + [0] * 4, dtype=I32)
    check(table, length, refs, 16, source=torch.tensor([9, -1, 2, 3], dtype=I32), need=torch.tensor([1, 1, 0, 0], dtype=I32))
    check(table, length, refs, 16, keep_len=torch.tensor([21, -1, 32, 4], dtype=I32), need=torch.tensor([1, 1, 1, -1], dtype=I32))
    check(table, length, refs, 16, need=torch.tensor([40, 0, 2 ** 31 - 1, 0], dtype=I32))


def test_in_a_graph():
    """A captured step, replayed: rows change in place, lengths by a copy behind it."""
    bs, B, M = 16, 3, 6
    table = torch.tensor([[0, 1, -1, -1, -1, -1], [2, -1, -1, -1, -1, -1], [3, 4, 5, -1, -1, -1]], dtype=I32)
    length, refs = torch.tensor([20, 16, 40], dtype=I32), torch.tensor([1] * 6 + [0] * 9, dtype=I32)
    need = torch.tensor([9, 9, 9], dtype=I32)
    t, n, r, d = table.cuda(), length.cuda(), refs.cuda(), need.cuda()
    out = dict(cache_len=torch.empty_like(n), row_status=torch.empty_like(n))
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        sv().spec_pages_update(t, n, r, block=bs, need=d, out=out)
        n.copy_(out["cache_len"] + 9)
    for _ in range(4):
        rows, lens, counts, status, _ = plain.pages(table, length, refs, bs, need=need)
        g.replay()
        torch.cuda.synchronize()
        assert t.tolist() == rows and r.tolist() == counts and out["row_status"].tolist() == status
        table, refs, length = torch.tensor(rows, dtype=I32), torch.tensor(counts, dtype=I32), torch.tensor(lens, dtype=I32) + 9
