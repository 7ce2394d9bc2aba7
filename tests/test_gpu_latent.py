"""The paged latent cache on the GPU against plain 64-bit forms: appending, attention (chain and tree masks, ragged and empty
sequences, strides, what is not finite where no row sees it), compaction, streams and graph capture."""

import math
import random

import pytest
import torch

import latent_plain as plain
from gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
SCALE = 192 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def sv():
    import speculative_decoding_verification_29_gb300 as m

    return m


def strided(x, how):
    """x [T, H, D] on the GPU: dense, heads outside tokens, or in rows that miss 16-byte boundaries."""
    if how == "heads":
        return x.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    if how == "odd":
        T, H, D = x.shape
        y = torch.zeros(max(1, T) * H * (D + 3) + 1, dtype=x.dtype, device="cuda").as_strided((T, H, D), (H * (D + 3), D + 3, 1), 1)
        y.copy_(x)
        return y
    return x.cuda()


def tree_mask(seed, B, n):
    rng = random.Random(seed)
    m = torch.zeros(B, n, n, dtype=torch.uint8)
    for b in range(B):
        for i in range(n):
            if i:
                m[b, i] = m[b, rng.randrange(i)]
            m[b, i, i] = 1
    return m


def queries(c, heads, seed, size=0.7):
    g = torch.Generator().manual_seed(seed + 77)
    return (torch.randn(sum(c.new), heads, c.C + c.R, generator=g) * size).to(c.dt)


def attend(c, q, args=None, scale=SCALE, mask=None, most=None, **kw):
    p, t, n = args or c.to("cuda")
    return sv().spec_latent_attention(q, p, t, n, c.cu.cuda(), max_tokens=most or max(max(c.new), 1), value_dim=c.C, sm_scale=scale,
                                      tree_mask=None if mask is None else mask.cuda(), **kw)


def close(got, want, tol, what=""):
    d = (got.double().cpu() - want).abs()
    assert not bool((d > tol).any()) and bool(torch.isfinite(got).all()), (what, float((d - tol).max()), float((d / (tol + 1e-30)).max()))


# --------------------------------------------------------------- attention --

ATTEND = [
    # ctx, new, heads, C, R, block, dtype, tree, strides, layout
    ([5, 0, 127, 128], [1, 1, 1, 1], 16, 512, 64, 16, BF, False, "dense", "dense"),
    ([700, 0, 63, 300], [1, 0, 1, 1], 1, 512, 64, 64, HF, False, "odd", "padded"),
    ([517], [1], 32, 512, 64, 16, BF, False, "heads", "dense"),
    ([900, 2], [3, 1], 11, 256, 32, 32, HF, False, "dense", "slots"),
    ([1500, 31, 64], [1, 1, 1], 48, 384, 48, 128, BF, False, "dense", "dense"),
    ([400, 130], [4, 3], 15, 128, 16, 16, HF, False, "odd", "dense"),
    ([300, 1], [9, 5], 7, 512, 64, 32, BF, False, "heads", "slots"),
    ([200, 0, 65], [13, 13, 13], 5, 512, 64, 64, HF, True, "dense", "dense"),
    # more than 64 rows
    ([300, 0, 129], [9, 9, 9], 16, 512, 64, 64, BF, False, "dense", "dense"),
    ([63, 64, 2], [9, 4, 9], 16, 512, 32, 16, HF, False, "odd", "padded"),
    ([700, 20, 0], [20, 1, 7], 20, 256, 64, 32, BF, False, "heads", "slots"),
    ([100, 350], [61, 61], 8, 512, 64, 128, HF, True, "dense", "dense"),
    ([50, 0], [30, 150], 3, 384, 16, 64, BF, False, "dense", "dense"),
    ([0, 90], [170, 40], 4, 128, 64, 16, HF, True, "dense", "dense"),
    ([1200], [1], 128, 512, 64, 64, BF, False, "dense", "dense"),
]


@pytest.mark.parametrize("ctx,new,heads,C,R,bs,dt,tree,how,layout", ATTEND)
def test_attention(ctx, new, heads, C, R, bs, dt, tree, how, layout):
    c = plain.Cache(ctx, new, C, R, bs, dt, seed=len(ctx) + C, layout=layout).fill()
    q = queries(c, heads, 3)
    mask = tree_mask(5, len(ctx), max(new)) if tree else None
    T = sum(new)
    out = strided(torch.full((T + 2, heads, C), 9.0, dtype=dt), how)
    status = torch.full((len(ctx) + 1,), 5, dtype=torch.int32, device="cuda")
    r = attend(c, strided(q, how), mask=mask, out=dict(out=out[1: T + 1], row_status=status))
    assert status.tolist() == [0] * len(ctx) + [5]
    want, tol = plain.attention(c, q, SCALE, mask)
    close(r["out"], want, tol)
    assert bool((out[0] == 9).all()) and bool((out[-1] == 9).all())  # rows before and behind the sequences'
    again = attend(c, strided(q, how), mask=mask)
    assert torch.equal(again["out"], r["out"])


@pytest.mark.parametrize("heads,dt", [(4, BF), (32, BF), (32, HF)])
@pytest.mark.parametrize("scale", [-SCALE, 0.0, 1e-30, 3.0])
def test_scales(heads, dt, scale):
    c = plain.Cache([70, 200], [5, 5], 512, 64, 32, dt, seed=1).fill()
    q = queries(c, heads, 4, 0.2)
    close(attend(c, q.cuda(), scale=scale)["out"], *plain.attention(c, q, scale), scale)


@pytest.mark.parametrize("heads", [4, 32])
@pytest.mark.parametrize("dt", [BF, HF])
def test_scores_that_rise(heads, dt):
    """Every tile's scores pass the last one's by far more than 2^8, or stay far below them."""
    c = plain.Cache([900, 900], [5, 5], 128, 16, 64, dt, seed=2).fill(0.05)
    q = queries(c, heads, 5, 0.05)
    q[..., 0] = 4.0
    for b in range(2):
        for t in range(900):
            blk, s = c.slot(b, t)
            c.pool[blk, s, 0] = (t // 64) * 30.0 * (1 if b == 0 else -1)
    close(attend(c, q.cuda(), scale=1.0)["out"], *plain.attention(c, q, 1.0))


@pytest.mark.parametrize("heads,n", [(5, 9), (20, 9), (8, 40), (2, 140)])
@pytest.mark.parametrize("dt", [BF, HF])
def test_what_no_row_sees(heads, n, dt):
    """Infinities and NaN in entries of the step that only some rows see, rows that see nothing, a mask of nothing."""
    bad = n // 2
    c = plain.Cache([130, 0], [n, n], 256, 32, 32, dt, seed=6).fill()
    q = queries(c, heads, 7)
    mask = tree_mask(8, 2, n)
    mask[:, :, bad] = 0
    mask[0, bad:, bad] = 1  # the second sequence's rows never see it
    mask[1, 1] = 0  # a row without anything
    for b, x in ((0, math.nan), (1, math.inf)):
        blk, s = c.slot(b, c.ctx[b] + bad)
        c.pool[blk, s, 3::7] = x
    r = attend(c, q.cuda(), mask=mask)
    assert r["row_status"].tolist() == [0, 0]
    clean = plain.Cache([130, 0], [n, n], 256, 32, 32, dt, seed=6).fill()
    sees = mask.clone()
    sees[0, bad:] = 0
    want, tol = plain.attention(clean, q, SCALE, sees)
    rows = torch.ones(2 * n, dtype=torch.bool)
    rows[bad:n] = False
    close(r["out"][rows.cuda()], want[rows], tol[rows])
    assert bool(torch.isnan(r["out"][bad:n]).all())
    assert bool((r["out"][n + 1] == 0).all())
    # under the causal mask, rows before the entry
    r = attend(c, q.cuda())
    want, tol = plain.attention(clean, q, SCALE)
    for b in range(2):
        close(r["out"][b * n: b * n + bad], want[b * n: b * n + bad], tol[b * n: b * n + bad])
        assert bool(torch.isnan(r["out"][b * n + bad: (b + 1) * n]).all())


@pytest.mark.parametrize("heads", [6, 24])
def test_bad_lengths_and_blocks(heads):
    c = plain.Cache([100, 50, 70, 10], [9, 9, 9, 9], 512, 64, 32, BF, seed=9).fill()
    q = queries(c, heads, 10)
    want, tol = plain.attention(c, q, SCALE)
    p, t, n = c.to("cuda")
    t[0, 3] = c.num  # the block of positions 96 .. 127: rows of sequence 0 see it
    t[1, 1] = -3  # 32 .. 63: the step's first rows see it too
    n[2] = -1
    r = attend(c, q.cuda(), (p, t, n))
    assert r["row_status"].tolist() == [64, 64, 64, 0]
    assert bool(torch.isnan(r["out"][:27]).all())
    close(r["out"][27:], want[27:], tol[27:])
    p, t, n = c.to("cuda")
    t[0, 3] = -1
    n[0] = 91  # tokens 0 .. 4 lie in 91 .. 95, before the missing block
    moved = plain.Cache([91, 50, 70, 10], [9, 9, 9, 9], 512, 64, 32, BF, seed=9)
    moved.pool, moved.table = c.pool, c.table
    want, tol = plain.attention(moved, q, SCALE)
    r = attend(c, q.cuda(), (p, t, n))
    assert r["row_status"].tolist() == [64, 0, 0, 0] and bool(torch.isnan(r["out"][5:9]).all())
    close(r["out"][:5], want[:5], tol[:5])
    cu = c.cu.clone()
    cu[2] = 3  # falls: sequence 1 is unsound
    r = sv().spec_latent_attention(q.cuda(), *c.to("cuda"), cu.cuda(), max_tokens=40, value_dim=512, sm_scale=SCALE)
    assert r["row_status"].tolist()[1] == 64


def test_long_context_and_many_sequences():
    c = plain.Cache([20001, 6], [2, 2], 512, 64, 128, BF, seed=11).fill()
    for heads in (3, 40):
        q = queries(c, heads, 12)
        close(attend(c, q.cuda())["out"], *plain.attention(c, q, SCALE))
    n = 700
    c = plain.Cache([i % 5 for i in range(n)], [1] * n, 128, 16, 16, HF, seed=13).fill()
    for heads in (2, 80):
        q = queries(c, heads, 14)
        close(attend(c, q.cuda())["out"], *plain.attention(c, q, SCALE))


def test_pool_beyond_4_gb():
    W, bs = 576, 128
    blocks = (5 << 30) // (W * bs * 2)
    pool = torch.zeros(blocks, bs, W, dtype=BF, device="cuda")
    c = plain.Cache([200], [3], 512, 64, bs, BF, seed=15).fill()
    pool[blocks - 2], pool[blocks - 5] = c.pool[c.table[0, 0]].cuda(), c.pool[c.table[0, 1]].cuda()
    t = torch.tensor([[blocks - 2, blocks - 5]], dtype=torch.int32, device="cuda")
    for heads in (8, 30):
        q = queries(c, heads, 16)
        close(attend(c, q.cuda(), (pool, t, c.len.cuda()))["out"], *plain.attention(c, q, SCALE))


@pytest.mark.parametrize("heads", [4, 24])
def test_graphs_and_streams(heads):
    """Two captured calls with workspaces of their own, replayed on refilled inputs; a call on another stream."""
    cs = [plain.Cache([300, 40], [9, 9], 512, 64, 32, BF, seed=20 + i).fill() for i in range(2)]
    qs = [queries(c, heads, 21 + i) for i, c in enumerate(cs)]
    args, dq = cs[0].to("cuda"), qs[0].cuda()
    cu = cs[0].cu.cuda()
    call = lambda **kw: sv().spec_latent_attention(dq, *args, cu, max_tokens=9, value_dim=512, sm_scale=SCALE, **kw)["out"]  # noqa: E731
    first = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, first)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        one, two = call(), call()
    for i in (1, 0):
        for a, b in zip(args, cs[i].to("cuda")):
            a.copy_(b)
        dq.copy_(qs[i].cuda())
        g.replay()
        torch.cuda.synchronize()
        close(one, *plain.attention(cs[i], qs[i], SCALE))
        assert torch.equal(one, two)


# ------------------------------------------------------------------ append --

APPEND = [
    # ctx, new, C, R, block, input type, cache type, interleaved, norm, heads, strides, layout
    ([5, 0, 31, 64], [9, 9, 9, 9], 512, 64, 16, BF, BF, False, True, 16, "dense", "dense"),
    ([0, 15, 16], [1, 1, 1], 256, 32, 16, HF, HF, True, True, 5, "odd", "padded"),
    ([3, 200], [130, 0], 384, 48, 64, torch.float32, BF, True, False, 3, "heads", "slots"),
    ([127, 0, 1], [300, 1, 2], 128, 16, 128, torch.float32, HF, False, True, 0, "dense", "dense"),
    ([0], [1], 512, 64, 32, BF, BF, False, False, 128, "odd", "dense"),
    ([40, 0, 0, 7], [0, 700, 0, 33], 512, 64, 32, HF, HF, False, True, 4, "dense", "dense"),
]


@pytest.mark.parametrize("ctx,new,C,R,bs,dt,cdt,inter,norm,heads,how,layout", APPEND)
@pytest.mark.parametrize("place", ["stored", "given"])
def test_append(ctx, new, C, R, bs, dt, cdt, inter, norm, heads, how, layout, place):
    c = plain.Cache(ctx, new, C, R, bs, cdt, seed=31, layout=layout)
    g = torch.Generator().manual_seed(32)
    T = sum(new)
    down = (torch.randn(T, C + R, generator=g) * 2).to(dt)
    q = torch.randn(T, max(heads, 1), C + R, generator=g).to(dt)
    w = torch.rand(C, generator=g) + 0.5
    w = w.to(dt) if heads != 5 else w
    freq = [10000.0 ** (-2 * i / R) for i in range(R // 2)]
    pos = torch.tensor([x + i for x, n in zip(ctx, new) for i in range(n)], dtype=torch.int32)
    if place == "given":
        pos = (pos * 7919 + 3) % 100003
    p, t, n = c.to("cuda")
    before = p.clone()
    x = strided(down[:, None], how)[:, 0]
    rows = strided(q, how)[..., C:] if heads else None
    r = sv().spec_latent_append(x[:, :C], x[:, C:], p, t, n, c.cu.cuda(), inv_freq=freq, interleaved=inter,
                                norm_weight=w.cuda() if norm else None, eps=1e-5, q_rope=rows,
                                positions=pos.cuda() if place == "given" else None)
    assert r["row_status"].tolist() == [0] * len(ctx)
    # fp32 arithmetic on a few operations and a sum of C squares of one sign; angles: 2^-32 of a turn and sincospif's 2^-22
    u, fine = plain.half_step(cdt), 64 * 2.0 ** -23
    y = plain.normalise(down[:, :C], w if norm else None, 1e-5)
    z = torch.stack([plain.rotate(down[i, C:], int(pos[i]), freq, inter) for i in range(T)])
    want = torch.cat((y, z), 1)
    size = torch.cat((y.abs(), down[:, C:].double().abs().amax(1, keepdim=True).expand(-1, R) * 2), 1)
    got, at = p.double().cpu(), 0
    touched = torch.zeros(p.shape[:2], dtype=torch.bool)
    for b, (k, m) in enumerate(zip(ctx, new)):
        for i in range(m):
            blk, s = c.slot(b, k + i)
            touched[blk, s] = True
            d = (got[blk, s] - want[at]).abs()
            assert bool((d <= u * want[at].abs() * (1 + fine) + fine * size[at] + (2.0 ** -25 if cdt == HF else 0)).all()), (b, i)
            at += 1
    same = p.view(torch.int16).cpu() == before.view(torch.int16).cpu() if p.is_contiguous() else \
        p.cpu().contiguous().view(torch.int16) == before.cpu().contiguous().view(torch.int16)
    assert bool(same[~touched].all())
    if heads:
        uq = plain.half_step(dt)
        wq = torch.stack([plain.rotate(q[i, :, C:], int(pos[i]), freq, inter) for i in range(T)])
        big = q[..., C:].double().abs().amax(-1, keepdim=True) * 2
        d = (r["q_out"].double().cpu() - wq).abs()
        assert bool((d <= uq * wq.abs() * (1 + fine) + fine * big + (2.0 ** -25 if dt == HF else 0)).all())
        keep = rows.clone()
        r2 = sv().spec_latent_append(x[:, :C], x[:, C:], p, t, n, c.cu.cuda(), inv_freq=freq, interleaved=inter, q_rope=keep,
                                     q_out=keep, positions=pos.cuda() if place == "given" else None)
        assert r2["q_out"] is keep and torch.equal(keep, r["q_out"])


def test_append_far_positions_zeros_and_bad_sequences():
    c = plain.Cache([40, 3, 50, 9], [4, 4, 4, 4], 128, 16, 16, BF, seed=33)
    x = torch.zeros(16, 144, dtype=BF)
    x[3:, 128:] = 1.5
    freq = [1.0 / (i + 1) for i in range(8)]
    p, t, n = c.to("cuda")
    t[1, 0] = 99  # a block outside the pool
    n[2] = -4
    before = p.clone()
    pos = torch.full((16,), (1 << 31) - 1, dtype=torch.int32)
    w = torch.ones(128)
    r = sv().spec_latent_append(x[:, :128].cuda(), x[:, 128:].cuda(), p, t, n, c.cu.cuda(), inv_freq=freq, positions=pos.cuda(),
                                norm_weight=w.cuda(), eps=1e-6)
    assert r["row_status"].tolist() == [0, 64, 64, 0]
    blk, s = c.slot(0, 43)
    assert bool((p[blk, s, :128] == 0).all())
    turns = [math.fmod(((1 << 31) - 1) * f, 2 * math.pi) for f in freq]
    want = torch.tensor([1.5 * (math.cos(a) - math.sin(a)) for a in turns] + [1.5 * (math.cos(a) + math.sin(a)) for a in turns])
    # the double product is off by 2^31 2^-53 of a radian
    assert bool(((p[blk, s, 128:].float().cpu() - want).abs() <= 2.0 ** -8 * want.abs() + 3e-6).all())
    for b in (1, 2):
        for i in range(4):
            j, s = c.slot(b, c.ctx[b] + i)
            if b == 2 or j != 99:
                assert torch.equal(p[j, s].view(torch.int16), before[j, s].view(torch.int16))


def test_append_of_shared_tokens():
    """Where cu_tokens falls, every sequence whose own range is sound gets all of its tokens."""
    c = plain.Cache([5, 7, 3], [6, 6, 6], 128, 32, 16, BF, seed=34)
    g = torch.Generator().manual_seed(35)
    x = torch.randn(10, 160, generator=g).to(BF)
    p, t, n = c.to("cuda")
    cu = torch.tensor([0, 6, 4, 9], dtype=torch.int32, device="cuda")  # sequence 1 is unsound, 0 and 2 share 4 and 5
    freq = [0.5 ** i for i in range(16)]
    r = sv().spec_latent_append(x[:, :128].cuda(), x[:, 128:].cuda(), p, t, n, cu, inv_freq=freq)
    assert r["row_status"].tolist() == [0, 64, 0]
    for b, lo, hi in ((0, 0, 6), (2, 4, 9)):
        for i in range(hi - lo):
            blk, s = c.slot(b, c.ctx[b] + i)
            assert torch.equal(p[blk, s, :128].cpu(), x[lo + i, :128])
            z = plain.rotate(x[lo + i, 128:], c.ctx[b] + i, freq, False)
            d = (p[blk, s, 128:].double().cpu() - z).abs()
            assert bool((d <= 2.0 ** -8 * z.abs() + 1e-4).all())


# ----------------------------------------------------------------- compact --


@pytest.mark.parametrize("planes", [0, 1, 5])
@pytest.mark.parametrize("bs,C,R,dt", [(16, 512, 64, BF), (64, 128, 16, HF)])
def test_compact(planes, bs, C, R, dt):
    ctx, N, D = [30, 0, 61, 17, 5, 9, 8], 40, 12
    c = plain.Cache(ctx, [N] * 7, C, R, bs, dt, seed=41).fill()
    rng = random.Random(42)
    path, acc = torch.full((7, D), -1, dtype=torch.int32), []
    for b in range(7):
        L = [11, 0, 5, 7, 3, 2, -1][b]
        row = [0] + sorted(rng.sample(range(1, N), max(L, 0)))
        path[b, : len(row)] = torch.tensor(row, dtype=torch.int32)
        acc.append(L)
    path[4, :4] = torch.tensor([0, 1, 2, 3])  # nothing moves
    path[5, :3] = torch.tensor([0, 4, 4])  # does not rise
    p, t, n = c.to("cuda")
    if planes:
        p = torch.stack([p.roll(i, 0) if i else p for i in range(planes)])
        p[:] = torch.randn(p.shape, generator=torch.Generator().manual_seed(43)).to(dt).cuda()
    want = p.clone()
    flat = want if planes else want[None]
    for b, L in enumerate(acc):
        if L < 0 or b == 5:
            continue
        moved = [flat[:, c.slot(b, ctx[b] + int(path[b, k]))[0], c.slot(b, ctx[b] + int(path[b, k]))[1]].clone() for k in range(L + 1)]
        for k, x in enumerate(moved):
            i, s = c.slot(b, ctx[b] + k)
            flat[:, i, s] = x
    a = torch.tensor(acc, dtype=torch.int32, device="cuda")
    r = sv().spec_latent_compact(p, t, n, a, path.cuda())
    assert r["new_len"].tolist() == [42, 1, 67, 25, 9, -1, -1]
    assert r["row_status"].tolist() == [0, 0, 0, 0, 0, 8, 0]
    assert torch.equal(p.view(torch.int16), want.view(torch.int16))
    r = sv().spec_latent_compact(p, t, n, a)
    assert r["new_len"].tolist() == [42, 1, 67, 25, 9, 12, -1] and torch.equal(p.view(torch.int16), want.view(torch.int16))
    t[0, 0] = -1
    t[0, (30 + int(path[0, 11])) // bs] = c.num
    assert sv().spec_latent_compact(p, t, n, a, path.cuda())["row_status"].tolist()[0] == 64


@pytest.mark.parametrize("heads", [16, 32])
def test_uneven_steps_that_add_up(heads):
    """As many tokens as B steps of max_tokens, but one sequence has fewer and one more than it may: its rows are NaN."""
    c = plain.Cache([140, 300, 77], [9, 3, 15], 512, 64, 32, BF, seed=50).fill()
    q = queries(c, heads, 51)
    want, tol = plain.attention(c, q, SCALE)
    r = attend(c, q.cuda(), most=9)
    assert r["row_status"].tolist() == [0, 0, 64]
    close(r["out"][:12], want[:12], tol[:12])
    assert bool(torch.isnan(r["out"][12:]).all())


def test_two_streams_at_once():
    """Calls of both kernels in flight on two streams, each with memory of its own."""
    c = plain.Cache([900, 40, 1500], [9, 9, 9], 512, 64, 32, BF, seed=52).fill()
    args = c.to("cuda")
    qs = [queries(c, h, 53).cuda() for h in (4, 24)]
    first = [attend(c, q, args)["out"] for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, (q, s) in enumerate(zip(qs, streams)):
            got[i].append(attend(c, q, args, stream=s)["out"])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, first[i]) for x in got[i])
