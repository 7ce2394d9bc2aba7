"""The 8-bit paged KV cache on the GPU against plain 64-bit forms: appending
with rotation, attention (chain and tree masks, ragged and empty sequences,
strides, garbage in places no row sees), compaction, row statuses, streams and
graph capture."""

import math
import random

import pytest
import torch

import kv8_plain as plain
from gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def sv():
    import speculative_decoding_verification_29_gb300 as m

    return m


def randn(g, *shape):
    return torch.randn(*shape, generator=g)


def strided(x, how, dev="cuda"):
    """x [T, H, D] on the GPU: dense, heads outside tokens, or in rows that miss 16-byte boundaries."""
    if how == "heads":
        return x.transpose(0, 1).contiguous().to(dev).transpose(0, 1)
    if how == "odd":
        y = torch.zeros(x.shape[0], x.shape[1] * (x.shape[2] + 3) + 1, dtype=x.dtype, device=dev)
        y = y.as_strided((x.shape[0], x.shape[1], x.shape[2]), (y.stride(0), x.shape[2] + 3, 1), 1)
        y.copy_(x)
        return y
    return x.to(dev)


# ------------------------------------------------------------------ append --

APPEND = [
    # ctx, new, H, D, block, dtype, rot, interleaved, strides, layout
    ([5, 0, 31, 64], [9, 9, 9, 9], 2, 128, 16, BF, 128, False, "dense", "hnd"),
    ([0, 15, 16, 17], [1, 1, 1, 1], 1, 64, 16, HF, 64, False, "dense", "hnd"),
    ([3, 200], [130, 0], 3, 128, 64, torch.float32, 64, True, "odd", "nhd"),
    ([127, 0, 1], [300, 1, 2], 2, 64, 128, BF, 32, False, "heads", "padded"),
    ([0], [1], 1, 128, 32, torch.float32, 0, False, "dense", "hnd"),
    ([40, 0, 0, 7], [0, 70, 0, 33], 2, 128, 32, HF, 128, True, "odd", "hnd"),
    ([100], [61], 8, 128, 64, BF, 16, False, "dense", "nhd"),
]


@pytest.mark.parametrize("ctx,new,H,D,bs,dt,rot,inter,how,layout", APPEND)
def test_append(ctx, new, H, D, bs, dt, rot, inter, how, layout):
    c = plain.Cache(ctx, new, H, D, bs, seed=sum(ctx) + D, layout=layout).fill(upto=ctx)
    T = sum(new)
    g = torch.Generator().manual_seed(1)
    k, v = (randn(g, T, H, D) * 2.0 ** randn(g, T, H, 1)).to(dt), (randn(g, T, H, D) * 3).to(dt)
    q = randn(g, T, 3, D).to(dt)
    freq = [10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)] if rot else None
    args = c.to("cuda")
    r = sv().spec_kv8_append(strided(k, how), strided(v, how), *args, c.cu.cuda(), inv_freq=freq, interleaved=inter,
                             q=strided(q, how))
    torch.cuda.synchronize()
    assert r["row_status"].tolist() == [0] * len(ctx)
    want, raw = plain.append(c, k, v, freq, inter)
    assert torch.equal(args[2].cpu(), want[2]) and torch.equal(args[3].cpu(), want[3])
    assert torch.equal(args[1].cpu(), want[1])  # values are not rotated: every code is the rounding's
    got = args[0].cpu()
    written = ~torch.isnan(raw[0])
    assert torch.equal(got[~written], want[0][~written])
    # rotated keys: the rotation's fp32 error (2^-22 of the pair's size) may move a value over a border, so each is
    # within half a step (2^-4 of the value, 2^-10 of the scale below the normal range) of the exact one
    val = got.view(torch.float8_e4m3fn).double()
    scale = torch.pow(2.0, want[2].double() - 127)[:, :, None, None]
    big = raw[0].abs().nan_to_num(0).amax(-1, keepdim=True)
    err = (val * scale - raw[0]).abs()
    assert (err <= torch.maximum(raw[0].abs() * 2.0 ** -4, scale * 2.0 ** -10) * (1 + 2.0 ** -10) + big * 2.0 ** -21)[written].all()
    wq = torch.stack([plain.rotate(q[t].double(), _pos(c, t), freq, inter) for t in range(T)])
    lim = wq.abs() * torch.finfo(dt).eps * 0.5 * 1.01 + wq.abs().amax(-1, keepdim=True) * 2.0 ** -21
    if dt == HF:
        lim = lim + 2.0 ** -25
    assert ((r["q_out"].cpu().double() - wq).abs() <= lim).all()


def _pos(c, t):
    b = int(torch.searchsorted(c.cu, torch.tensor(t, dtype=torch.int32), right=True)) - 1
    return c.ctx[b] + t - int(c.cu[b])


def test_append_far_positions_and_tree_positions():
    """Rotation by given positions up to 2^31 - 1 keeps fp32 accuracy."""
    c = plain.Cache([0, 20], [6, 6], 1, 128, 16)
    g = torch.Generator().manual_seed(2)
    k, v = randn(g, 12, 1, 128), randn(g, 12, 1, 128)
    pos = torch.tensor([0, 1, 4097, 1000003, 2 ** 30 + 7, 2 ** 31 - 1] * 2, dtype=torch.int32)
    freq = [1000000.0 ** (-2.0 * i / 128) for i in range(64)]
    q = randn(g, 12, 2, 128)
    r = sv().spec_kv8_append(k.cuda(), v.cuda(), *c.to("cuda"), c.cu.cuda(), inv_freq=torch.tensor(freq, dtype=torch.float64),
                             positions=pos.cuda(), q=q.cuda())
    wq = torch.stack([plain.rotate(q[t].double(), int(pos[t]), freq, False) for t in range(12)])
    # 64-bit angles themselves are good to 2^-53 of 2^31 radians: 2^-22; the fp32 turn adds 2^-22
    assert (r["q_out"].cpu().double() - wq).abs().max() <= 4 * 2.0 ** -21


def test_append_turns_backwards():
    """Frequencies and positions below zero: turning by (-f, p) is turning by (f, -p), bit for bit, and right."""
    c = plain.Cache([0], [5], 1, 128, 16)
    g = torch.Generator().manual_seed(4)
    k, q = randn(g, 5, 1, 128), randn(g, 5, 2, 128)
    pos = torch.tensor([1, 3, 1000, 10 ** 6 + 1, 2 ** 31 - 1], dtype=torch.int32)
    freq = [10.0 ** (-i / 4.0) for i in range(64)]  # down to 1.8e-16
    a, b = (sv().spec_kv8_append(k.cuda(), k.cuda(), *c.to("cuda"), c.cu.cuda(), inv_freq=[s * f for f in freq],
                                 positions=(-s * pos).cuda(), q=q.cuda())["q_out"].cpu() for s in (1, -1))
    assert torch.equal(a, b)
    wq = torch.stack([plain.rotate(q[t].double(), -int(pos[t]), freq, False) for t in range(5)])
    assert (a.double() - wq).abs().max() <= 4 * 2.0 ** -21


def test_append_special_values():
    """Zeros, infinities, NaN, and magnitudes outside the scales' range."""
    c = plain.Cache([0, 3], [8, 2], 2, 64, 16).fill(upto=[0, 3])
    g = torch.Generator().manual_seed(3)
    k, v = randn(g, 10, 2, 64), randn(g, 10, 2, 64)
    k[0, 0] = 0.0
    k[1, 0, 5], k[2, 0, 6], k[3, 0, 7] = math.inf, -math.inf, math.nan
    v[:8, 0] = 0.0
    v[:8, 1] *= 1e-20
    v[8, 0, 1], k[9, 1, 2] = 3e38, math.inf
    args = c.to("cuda")
    sv().spec_kv8_append(k.cuda(), v.cuda(), *args, c.cu.cuda())
    want, _ = plain.append(c, k, v)
    for i in range(4):
        assert torch.equal(args[i].cpu(), want[i]), i


def test_append_twice_is_append():
    """A step's second append (a retried step) leaves the same cache."""
    c = plain.Cache([37, 5], [9, 30], 2, 128, 32).fill(upto=[37, 5])
    g = torch.Generator().manual_seed(4)
    k, v = (randn(g, 39, 2, 128) * 9).to(BF), (randn(g, 39, 2, 128) * 9).to(BF)
    args = c.to("cuda")
    sv().spec_kv8_append(k.cuda(), v.cuda(), *args, c.cu.cuda())
    once = [a.clone() for a in args[:4]]
    sv().spec_kv8_append(k.cuda(), v.cuda(), *args, c.cu.cuda())
    assert all(torch.equal(a, b) for a, b in zip(args[:4], once))


def test_append_row_status():
    """Sequences with lengths or block ids out of range are reported and write nothing outside their blocks."""
    c = plain.Cache([10, 10, 10, 10], [4, 4, 4, 4], 1, 64, 16).fill()
    args = c.to("cuda")
    table, length = args[4], args[5]
    table[1, 0] = c.num  # one past the pool
    length[2] = -1
    length[3] = table.shape[1] * 16 - 2  # the table is too short for four more
    table[3] = table[3].clamp(min=0)
    before = [a.clone() for a in args[:4]]
    g = torch.Generator().manual_seed(5)
    k = randn(g, 16, 1, 64).cuda()
    r = sv().spec_kv8_append(k, k, *args, c.cu.cuda())
    assert r["row_status"].tolist() == [0, 64, 64, 64]
    i = int(table[0, 0])
    for a, b in zip(args[:4], before):
        same = torch.ones(c.num, dtype=torch.bool, device="cuda")
        same[i] = False
        assert torch.equal(a[same], b[same])
    bad = torch.tensor([0, 4, 2, 5, 99], dtype=torch.int32, device="cuda")  # falls, and passes T
    args = c.to("cuda")
    r = sv().spec_kv8_append(k, k, *args, bad)
    assert r["row_status"].tolist() == [0, 64, 0, 64]


# --------------------------------------------------------------- attention --

ATTN = [
    # ctx, new, Hq, H, D, block, dtype, tree, strides, layout
    ([0], [1], 1, 1, 128, 16, BF, False, "dense", "hnd"),
    ([517], [1], 32, 8, 128, 16, BF, False, "dense", "hnd"),
    ([0, 1, 127, 128, 129, 300], [1, 1, 1, 1, 1, 1], 8, 2, 128, 32, HF, False, "dense", "nhd"),
    ([100, 0, 255, 64], [9, 9, 9, 0], 8, 2, 128, 64, BF, False, "heads", "hnd"),
    ([33, 400], [9, 5], 14, 2, 128, 128, HF, False, "odd", "padded"),
    ([70, 5], [17, 16], 6, 2, 128, 16, BF, False, "dense", "hnd"),
    ([90, 0, 30], [61, 61, 61], 8, 2, 128, 32, BF, True, "dense", "hnd"),
    ([10, 250], [64, 64], 16, 2, 128, 64, HF, True, "heads", "nhd"),
    ([0, 40], [150, 131], 4, 2, 128, 64, BF, False, "dense", "hnd"),
    ([2500], [3], 4, 1, 128, 128, BF, False, "dense", "hnd"),
    ([3000, 17], [2, 1], 4, 4, 128, 16, HF, False, "dense", "hnd"),
    ([0, 1, 129, 700], [1, 2, 1, 9], 4, 2, 64, 32, HF, False, "dense", "hnd"),
    ([300, 20], [20, 20], 8, 2, 64, 16, BF, True, "odd", "nhd"),
    ([100], [140], 4, 1, 64, 128, BF, False, "heads", "padded"),
    ([260], [2], 64, 1, 128, 64, BF, False, "dense", "hnd"),
    # row tiles with one or two rows beside full ones
    ([0, 300, 5], [1, 70, 2], 2, 2, 128, 64, BF, False, "dense", "hnd"),
    ([20, 300, 0], [1, 70, 3], 4, 2, 64, 32, HF, False, "dense", "hnd"),
    ([130, 3], [257, 1], 1, 1, 128, 64, HF, False, "dense", "hnd"),
    ([9], [129], 4, 2, 64, 16, BF, False, "dense", "nhd"),
    ([700, 40, 0], [129, 128, 1], 1, 1, 64, 128, HF, False, "dense", "hnd"),
]


def run_attention(c, q, scale, tree, how="dense", **kw):
    args = c.to("cuda")
    r = sv().spec_kv8_attention(strided(q, how), *args, c.cu.cuda(), max_tokens=max(max(c.new), 1) if tree is None else
                                tree.shape[1], sm_scale=scale, tree_mask=None if tree is None else tree.cuda(), **kw)
    torch.cuda.synchronize()
    return r["out"].cpu().double(), r["row_status"].tolist()


def check_attention(c, q, tree=None, how="dense", scale=None):
    scale = c.D ** -0.5 if scale is None else scale
    got, status = run_attention(c, q, scale, tree, how)
    want, tol = plain.attention(c, q, scale, tree)
    assert status == [0] * len(c.ctx)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    fine = ~torch.isnan(want)
    bad = ((got - want).abs() > tol)[fine]
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {float(((got - want).abs() / tol)[fine].max()):.2f} tolerances"


@pytest.mark.parametrize("ctx,new,Hq,H,D,bs,dt,tree,how,layout", ATTN)
def test_attention(ctx, new, Hq, H, D, bs, dt, tree, how, layout):
    c = plain.Cache(ctx, new, H, D, bs, seed=len(ctx) + Hq, layout=layout).fill()
    g = torch.Generator().manual_seed(7)
    q = (randn(g, sum(new), Hq, D) * 2).to(dt)
    mask = plain.tree_mask(random.Random(1), len(ctx), max(new))[0] if tree else None
    check_attention(c, q, mask, how)


@pytest.mark.parametrize("new,Hq,H,D,dt", [((1, 2), 8, 4, 128, BF), ((5, 9), 12, 4, 64, HF), ((9, 16), 32, 4, 128, BF),
                                           ((9, 16), 32, 4, 64, HF), ((33, 61), 16, 2, 128, HF)])
def test_attention_many_items(new, Hq, H, D, dt):
    """Several items to a thread block, of odd and even numbers of tiles, some cut by a block's run."""
    rng = random.Random(5)
    B = 14 if new[1] < 30 else 6
    ctx = [rng.choice([rng.randint(0, 500), rng.randint(500, 2600)]) for _ in range(B)]
    c = plain.Cache(ctx, [rng.randint(*new) for _ in ctx], H, D, 64, seed=17).fill()
    g = torch.Generator().manual_seed(15)
    check_attention(c, (randn(g, sum(c.new), Hq, D) * 2).to(dt))


@pytest.mark.parametrize("new,Hq,H", [((1, 3), 2, 2), ((0, 9), 8, 1), ((3, 20), 16, 1), ((17, 34), 8, 1)])
def test_attention_short_items(new, Hq, H):
    """More thread blocks than tiles, and runs that end between an item's start and its first tile."""
    rng = random.Random(6)
    B = 90 if new[1] < 20 else 40
    c = plain.Cache([rng.choice([0, rng.randint(0, 127), rng.randint(0, 300)]) for _ in range(B)],
                    [rng.randint(*new) for _ in range(B)], H, 128, 32, seed=18).fill()
    check_attention(c, randn(torch.Generator().manual_seed(16), sum(c.new), Hq, 128).to(BF))


@pytest.mark.parametrize("dt", [BF, HF])
def test_attention_sharp_and_flat_weights(dt):
    """One entry that takes nearly all of the weight, then hundreds that share it, and the reverse."""
    c = plain.Cache([600, 600], [2, 2], 1, 128, 64, seed=3).fill(spread=0.2)
    q = torch.zeros(4, 2, 128, dtype=torch.float64)
    for b in range(2):
        k = c.rows(c.k, c.ks, b, 602)[0][0]
        top = k[5 if b == 0 else 590]
        q[2 * b: 2 * b + 2, 0] = top * 3.0
        q[2 * b: 2 * b + 2, 1] = top * 0.01
    check_attention(c, q.to(dt))


def test_attention_block_scales_far_apart():
    """Blocks whose scales differ by 2^30: the large values decide the result, the small keys the weights."""
    c = plain.Cache([300], [4], 2, 128, 16, seed=9).fill(spread=0.1)
    c.vs[c.table[0, :10].long()] -= 20
    c.vs[c.table[0, 12].long()] += 10
    c.ks[c.table[0, 3].long()] += 3
    g = torch.Generator().manual_seed(8)
    check_attention(c, randn(g, 4, 2, 128).to(BF))


def test_attention_empty_rows_and_unseen_garbage():
    """Rows whose mask leaves nothing give 0; NaN entries reach the rows that see them, and no others."""
    N = 12
    c = plain.Cache([0, 130], [N, N], 2, 128, 16, seed=5).fill()
    mask, _ = plain.tree_mask(random.Random(2), 2, N)
    mask[0, 3] = 0
    mask[0, :, 5] = 0
    mask[0, 5, 5] = 1  # node 5 is seen by itself alone
    mask[1, :, 7] = 0
    mask[1, 7, 7] = 1
    i = int(c.table[0, 0])
    c.v[i, 0, 5, 9] = 0x7F
    c.k[i, 1, 5, 3] = 0xFF
    j, s = int(c.table[1, (130 + 7) // 16]), (130 + 7) % 16
    c.v[j, 1, s, 100] = 0xFF
    g = torch.Generator().manual_seed(9)
    q = randn(g, 2 * N, 4, 128).to(BF)
    check_attention(c, q, mask)
    got, _ = run_attention(c, q, 128 ** -0.5, mask)
    assert (got[3] == 0).all()
    assert torch.isnan(got[5, :2, 9]).all() and torch.isnan(got[5, 2:]).all() and int(torch.isnan(got).sum()) == 2 + 2 * 128 + 2


def test_attention_nan_queries_stay_in_their_rows():
    c = plain.Cache([50], [3], 1, 128, 16, seed=6).fill()
    g = torch.Generator().manual_seed(10)
    q = randn(g, 3, 2, 128).to(BF)
    q[1, 0, 4] = math.nan
    got, _ = run_attention(c, q, 128 ** -0.5, None)
    assert torch.isnan(got[1, 0]).all() and int(torch.isnan(got).sum()) == 128


def test_attention_large_scores():
    """Scores of thousands, of both signs."""
    c = plain.Cache([200], [5], 1, 128, 32, seed=12).fill(spread=0.1)
    g = torch.Generator().manual_seed(11)
    q = (randn(g, 5, 2, 128) * 100).to(BF)
    got, _ = run_attention(c, q, 0.5, None)
    w = torch.einsum("tad,sd->tas", q.double(), c.rows(c.k, c.ks, 0, 205)[0][0]) * 0.5
    w = w.masked_fill(~(torch.arange(205) <= 200 + torch.arange(5)[:, None])[:, None, :], -math.inf)
    gap = w.topk(2, -1).values
    sure = (gap[..., 0] - gap[..., 1]) > 30  # one entry has all of the weight
    assert sure.sum() >= 5
    v = c.rows(c.v, c.vs, 0, 205)[0][0][w.argmax(-1)]
    assert ((got - v).abs() <= v.abs() * 2.0 ** -7)[sure].all()


def test_attention_row_status():
    c = plain.Cache([40, 40, 40, 40], [2, 2, 2, 2], 1, 128, 16, seed=4).fill()
    g = torch.Generator().manual_seed(12)
    q = randn(g, 8, 2, 128).to(BF)
    want, tol = plain.attention(c, q, 0.1)
    args = c.to("cuda")
    args[4][1, 1], args[4][2, 0] = -1, c.num
    args[5][3] = -5
    r = sv().spec_kv8_attention(q.cuda(), *args, c.cu.cuda(), max_tokens=2, sm_scale=0.1)
    assert r["row_status"].tolist() == [0, 64, 64, 64]
    got = r["out"].cpu().double()
    assert torch.isnan(got[2:]).all() and ((got[:2] - want[:2]).abs() <= tol[:2]).all()
    args = c.to("cuda")
    r = sv().spec_kv8_attention(q.cuda(), *args, c.cu.cuda(), max_tokens=1, sm_scale=0.1)
    assert r["row_status"].tolist() == [64] * 4 and torch.isnan(r["out"]).all()
    bad = torch.tensor([0, 2, 1, 8, 9], dtype=torch.int32, device="cuda")
    r = sv().spec_kv8_attention(q.cuda(), *args, bad, max_tokens=8, sm_scale=0.1)
    assert r["row_status"].tolist() == [0, 64, 0, 64]


def test_attention_no_tokens():
    c = plain.Cache([40, 3], [0, 0], 1, 128, 16).fill()
    r = sv().spec_kv8_attention(torch.empty(0, 2, 128, dtype=BF, device="cuda"), *c.to("cuda"), c.cu.cuda(), max_tokens=1)
    assert r["out"].shape == (0, 2, 128) and r["row_status"].tolist() == [0, 0]


def test_cache_beyond_32_bit_offsets():
    """A pool whose far blocks lie past 4 GB: the same entries there and at its start give the same result."""
    c = plain.Cache([100], [3], 2, 128, 64, seed=8, extra_blocks=0).fill()
    num = (9 << 29) // (2 * 64 * 128)
    far = [num - 1 - i for i in range(c.num)]
    big = [torch.empty(num, 2, 64, 128, dtype=torch.uint8, device="cuda") for _ in range(2)]
    sc = [torch.empty(num, 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
    table = c.table.clone()
    for i, f in enumerate(far):
        big[0][f], big[1][f] = c.k[i].cuda(), c.v[i].cuda()
        sc[0][f], sc[1][f] = c.ks[i].cuda(), c.vs[i].cuda()
        table[c.table == i] = f
    g = torch.Generator().manual_seed(13)
    q = randn(g, 3, 4, 128).to(BF)
    near = sv().spec_kv8_attention(q.cuda(), *c.to("cuda"), c.cu.cuda(), max_tokens=3)["out"]
    args = [*big, *sc, table.cuda(), c.len.cuda()]
    assert torch.equal(sv().spec_kv8_attention(q.cuda(), *args, c.cu.cuda(), max_tokens=3)["out"], near)
    k = randn(g, 3, 2, 128).to(BF).cuda()
    small = c.to("cuda")
    sv().spec_kv8_append(k, k, *small, c.cu.cuda())
    sv().spec_kv8_append(k, k, *args, c.cu.cuda())
    for i, f in enumerate(far):
        assert torch.equal(big[0][f], small[0][i]) and torch.equal(big[1][f], small[1][i])


# ----------------------------------------------------------------- compact --


@pytest.mark.parametrize("H,D,bs,layout", [(2, 128, 16, "hnd"), (3, 64, 32, "nhd"), (1, 128, 128, "padded"), (2, 64, 64, "hnd")])
def test_compact(H, D, bs, layout):
    N = 40
    ctx = [0, 7, 64, 100, 33]
    c = plain.Cache(ctx, [N] * 5, H, D, bs, seed=bs, layout=layout).fill(spread=2.0)
    path = torch.tensor([[0, 1, 5, 20, 39, -1], [0, 2, 3, 4, 30, 31], [0, 39, -1, -1, -1, -1], [0, -1, -1, -1, -1, -1],
                         [0, 1, 2, 3, 4, 5]], dtype=torch.int32)
    acc = torch.tensor([4, 5, 1, 0, 5], dtype=torch.int32)
    args = c.to("cuda")
    r = sv().spec_kv8_compact(*args, acc.cuda(), path.cuda())
    want = plain.compact(c, path, acc)
    assert r["row_status"].tolist() == [0] * 5 and r["new_len"].tolist() == [x + int(a) + 1 for x, a in zip(ctx, acc)]
    for i in range(4):
        assert torch.equal(args[i].cpu(), want[i]), i


def test_compact_long_path():
    c = plain.Cache([13], [130], 1, 128, 16, seed=2).fill(spread=1.5)
    path = torch.tensor([[0] + list(range(2, 127, 2))[:63]], dtype=torch.int32)
    acc = torch.tensor([63], dtype=torch.int32)
    args = c.to("cuda")
    sv().spec_kv8_compact(*args, acc.cuda(), path.cuda())
    for got, want in zip(args[:4], plain.compact(c, path, acc)):
        assert torch.equal(got.cpu(), want)


def test_compact_planes_and_chain():
    cs = [plain.Cache([7, 30], [20, 20], 2, 64, 16, seed=1).fill(spread=1.0)]
    for s in (2, 3):
        n = plain.Cache([7, 30], [20, 20], 2, 64, 16, seed=1)
        n.g.manual_seed(s)
        cs.append(n.fill(spread=1.0))
    path = torch.tensor([[0, 3, 9, 19], [0, 1, 18, -1]], dtype=torch.int32)
    acc = torch.tensor([3, 2], dtype=torch.int32)
    st = [torch.stack([x.to("cuda")[i] for x in cs]) for i in range(4)]
    r = sv().spec_kv8_compact(*st, cs[0].table.cuda(), cs[0].len.cuda(), acc.cuda(), path.cuda())
    assert r["new_len"].tolist() == [11, 33]
    for p, c in enumerate(cs):
        for i, want in enumerate(plain.compact(c, path, acc)):
            assert torch.equal(st[i][p].cpu(), want)
    before = [x.clone() for x in st]
    r = sv().spec_kv8_compact(*st, cs[0].table.cuda(), cs[0].len.cuda(), acc.cuda())
    assert r["new_len"].tolist() == [11, 33] and all(torch.equal(a, b) for a, b in zip(st, before))


def test_compact_row_status():
    N, D1 = 10, 4
    c = plain.Cache([5] * 7, [N] * 7, 1, 64, 16, seed=2).fill()
    path = torch.tensor([[1, 2, -1, -1], [0, 2, 2, -1], [0, 3, 1, -1], [0, 1, 2, 3], [0, 1, 999, -1], [0, 1, -1, -1],
                         [0, 2, 9, -1]], dtype=torch.int32)
    acc = torch.tensor([1, 2, 2, 4, 2, -1, 2], dtype=torch.int32)
    args = c.to("cuda")
    args[4][6, 0] = -3
    before = [a.clone() for a in args[:4]]
    r = sv().spec_kv8_compact(*args, acc.cuda(), path.cuda())
    assert r["row_status"].tolist() == [8, 8, 8, 8, 8, 0, 64] and r["new_len"].tolist() == [-1] * 7
    assert all(torch.equal(a, b) for a, b in zip(args[:4], before))
    assert path.shape[1] == D1


# --------------------------------------------------------- streams and graphs --


def _step_inputs(seed=21):
    c = plain.Cache([200, 77, 0], [9, 9, 9], 2, 128, 64, seed=seed).fill(upto=[200, 77, 0])
    g = torch.Generator().manual_seed(seed)
    return c, (randn(g, 27, 2, 128)).to(BF).cuda(), (randn(g, 27, 2, 128)).to(BF).cuda(), randn(g, 27, 8, 128).to(BF).cuda()


def _step(args, cu, k, v, q, freq, **kw):
    r = sv().spec_kv8_append(k, v, *args, cu, inv_freq=freq, q=q, **kw)
    return sv().spec_kv8_attention(r["q_out"], *args, cu, max_tokens=9, **kw)["out"]


def test_side_stream():
    """Calls on a stream that is not the current one: the temporaries are not reused early."""
    freq = [10000.0 ** (-2.0 * i / 128) for i in range(64)]
    c, k, v, q = _step_inputs()
    args, cu = c.to("cuda"), c.cu.cuda()
    want = _step(args, cu, k, v, q, freq)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    args2 = c.to("cuda")
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        outs.append(_step(args2, cu, k, v, q, freq, stream=s))
        torch.full((1 << 22,), 7, dtype=torch.uint8, device="cuda")  # the current stream takes freed memory at once
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_graph_capture():
    """Append and attention captured once, replayed on new inputs and lengths in the same buffers."""
    freq = [10000.0 ** (-2.0 * i / 128) for i in range(64)]
    c, k, v, q = _step_inputs(22)
    args, cu = c.to("cuda"), c.cu.cuda()
    _step(args, cu, k, v, q, freq)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = _step(args, cu, k, v, q, freq)
    c2, k2, v2, q2 = _step_inputs(23)
    c2.len[1] = 60  # shorter than before
    fresh = c2.to("cuda")
    want = _step(fresh, cu, k2, v2, q2, freq)
    for a, b in zip(args[:4] + args[5:] + [k, v, q], c2.to("cuda")[:4] + c2.to("cuda")[5:] + [k2, v2, q2]):
        a.copy_(b)
    args[4].copy_(c2.table)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_results_repeat():
    """The split of long contexts adds in a fixed order: results repeat bit for bit."""
    c = plain.Cache([5000, 1200], [9, 9], 2, 128, 64, seed=30).fill()
    g = torch.Generator().manual_seed(14)
    q = randn(g, 18, 8, 128).to(BF).cuda()
    args = c.to("cuda")
    first = sv().spec_kv8_attention(q, *args, c.cu.cuda(), max_tokens=9)["out"]
    for _ in range(10):
        assert torch.equal(sv().spec_kv8_attention(q, *args, c.cu.cuda(), max_tokens=9)["out"], first)
