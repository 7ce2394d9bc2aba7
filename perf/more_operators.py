"""Performance cases of the paged latent cache (one shared latent vector a token) and of the pages under it.

The cache of one layer is a pool of blocks in 16 bits, [blocks, block, C + R]: a token's slot holds its latent vector of C
dimensions, from which keys and values of every head come, and R rotated dimensions that the heads' keys share.
`block_table[b]` lists the blocks of sequence b in order; it has `cache_len[b]` tokens in the cache before the step, and the
step adds tokens cu_tokens[b] .. cu_tokens[b + 1] - 1 of the packed inputs after them. `refs[i]` counts the sequences that
hold block i; 0 is a free block.

`run` computes the operators in elementary torch operations (`own` false) or through the package (`own` true):
  append     normalises and rotates the step's latent vectors into the pool, and rotates its queries' last R dimensions
  attention  of queries that the keys' projection was absorbed into, all heads over the same slots, values: the C dimensions
  compact    moves the entries of an accepted path behind the context, in every layer
  pages      keeps each sequence's first tokens (of its own or of another sequence, which forks it), gives the blocks behind
             them back, and takes free blocks for the next step; a partly filled block that others share is copied
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SM_SCALE = (128 + 64) ** -0.5  # of the heads' keys before the projection was absorbed
CACHE_BAD = 64  # row_status of a sequence whose blocks did not suffice


def listed():
    return [
        # one user, one token on a short context: the latency of a single decode step
        _attention("attn_decode_one", B=1, new_lo=1, new_hi=1, ctx_lo=517, ctx_hi=517, block=16, heads=16),
        # a full decode batch on ragged contexts
        _attention("attn_decode", B=64, new_lo=1, new_hi=1, ctx_lo=1500, ctx_hi=6500, block=64),
        # the target's pass over K = 8 draft tokens and the root, the chain verification batch
        _attention("attn_verify", B=64, new_lo=9, new_hi=9, ctx_lo=1500, ctx_hi=6500, block=64),
        # the target's pass over merged trees of N = 61 nodes, fp16
        _attention("attn_tree", B=16, new_lo=61, new_hi=61, ctx_lo=500, ctx_hi=3500, block=32, heads=16, dtype="fp16",
                   tree=True),
        # two users with long contexts, K = 8, all 128 heads
        _attention("attn_long", B=2, new_lo=9, new_hi=9, ctx_lo=110001, ctx_hi=131072, block=128, heads=128),
        # prompts of several users after a shared prefix, a smaller latent vector, an odd number of heads
        _attention("attn_prompt", B=3, new_lo=500, new_hi=1500, ctx_lo=1, ctx_hi=1000, block=64, heads=20, latent=256,
                   rot=32),
        # the verification batch: normalised, rotated, with the queries of 32 heads
        _append("append_verify", B=64, new_lo=9, new_hi=9, ctx_lo=1500, ctx_hi=6500, block=64),
        # prompts, ragged, interleaved pairs
        _append("append_prompt", B=8, new_lo=1500, new_hi=4096, ctx_lo=0, ctx_hi=1000, block=64, heads=16,
                interleaved=True, dtype="fp16"),
        # accepted tree paths of one user, one layer
        _compact("compact_one", B=1, nodes=61, planes=1, ctx_lo=517, ctx_hi=517, block=16),
        # accepted tree paths of the tree batch in every one of 32 layers
        _compact("compact_tree", B=16, nodes=61, planes=32, ctx_lo=180, ctx_hi=420, block=64),
        # after a verification step of the batch: drop what was rejected, take blocks for the next nine tokens
        _pages("pages_step", B=64, nodes=9, planes=1, ctx_lo=1500, ctx_hi=6500, block=64),
        # four prompts sampled sixteen times each: forked, and every last block copied in all of 32 layers
        _pages("pages_fork", B=64, nodes=9, planes=32, ctx_lo=180, ctx_hi=1500, block=64, leaders=4),
    ]


def _attention(name, *, B, new_lo, new_hi, ctx_lo, ctx_hi, block, heads=32, latent=512, rot=64, dtype="bf16", tree=False):
    return dict(name=name, op="attention", B=B, new_lo=new_lo, new_hi=new_hi, ctx_lo=ctx_lo, ctx_hi=ctx_hi, block=block,
                heads=heads, latent=latent, rot=rot, dtype=dtype, tree=tree)


def _append(name, *, B, new_lo, new_hi, ctx_lo, ctx_hi, block, heads=32, latent=512, rot=64, dtype="bf16",
            interleaved=False, norm=True):
    return dict(name=name, op="append", B=B, new_lo=new_lo, new_hi=new_hi, ctx_lo=ctx_lo, ctx_hi=ctx_hi, block=block,
                heads=heads, latent=latent, rot=rot, dtype=dtype, interleaved=interleaved, norm=norm)


def _compact(name, *, B, nodes, planes, ctx_lo, ctx_hi, block, latent=512, rot=64, dtype="bf16"):
    return dict(name=name, op="compact", B=B, nodes=nodes, planes=planes, ctx_lo=ctx_lo, ctx_hi=ctx_hi, block=block,
                latent=latent, rot=rot, dtype=dtype)


def _pages(name, *, B, nodes, planes, ctx_lo, ctx_hi, block, leaders=0, latent=512, rot=64, dtype="bf16"):
    return dict(name=name, op="pages", B=B, nodes=nodes, planes=planes, ctx_lo=ctx_lo, ctx_hi=ctx_hi, block=block,
                leaders=leaders, latent=latent, rot=rot, dtype=dtype)


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the listed ones' ranges: decode, verification, tree, long and prompt attention, appends, compactions, steps
    and forks of the pages."""
    op = rng.choice(["attention"] * 4 + ["append"] * 2 + ["compact"] + ["pages"] * 2)
    block = rng.choice([16, 32, 64, 128])
    latent, rot = rng.choice([(512, 64), (512, 64), (256, 64), (256, 32), (128, 32)])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "attention":
        kind = rng.choice(["decode", "verify", "verify", "tree", "long", "prompt"])
        heads = rng.choice([1, 5, 8, 16, 16, 20, 32, 32, 64, 128])
        B, new, ctx = _log(rng, 1, 64), (1, 1), _log(rng, 16, 6500)
        if kind == "verify":
            K1 = rng.randint(2, 17)
            new = (rng.randint(1, K1), K1)
            heads = min(heads, 64)
        elif kind == "tree":
            B, new, ctx = _log(rng, 1, 16), (rng.randint(5, 64),) * 2, _log(rng, 16, 3500)
            heads = min(heads, 32)
        elif kind == "long":
            B, new, ctx = rng.randint(1, 2), (1, rng.randint(1, 9)), _log(rng, 20000, 131072)
        elif kind == "prompt":
            top = _log(rng, 65, 1500)
            B, new, ctx = rng.randint(1, 3), (top // 2, top), _log(rng, 1, 1000)
            heads = min(heads, 20)
        case = _attention("", B=B, new_lo=new[0], new_hi=new[1], ctx_lo=ctx // 3, ctx_hi=ctx, block=block, heads=heads,
                          latent=latent, rot=rot, dtype=dtype, tree=kind == "tree")
    elif op == "append":
        prompt = rng.random() < 0.4
        top = _log(rng, 65, 4096) if prompt else rng.randint(1, 61)
        B = rng.randint(1, 8) if prompt else _log(rng, 1, 64)
        ctx = _log(rng, 1, 6500)
        case = _append("", B=B, new_lo=max(1, top // 2), new_hi=top, ctx_lo=ctx // 3, ctx_hi=ctx, block=block,
                       heads=rng.choice([0, 5, 16, 32]), latent=latent, rot=rot, dtype=dtype,
                       interleaved=rng.random() < 0.5, norm=rng.random() < 0.7)
    elif op == "compact":
        ctx = _log(rng, 16, 420)
        case = _compact("", B=_log(rng, 1, 16), nodes=rng.randint(9, 64), planes=_log(rng, 1, 32), ctx_lo=ctx // 3,
                        ctx_hi=ctx, block=block, latent=latent, rot=rot, dtype=dtype)
    else:
        fork = rng.random() < 0.5
        B, ctx = _log(rng, 2 if fork else 1, 64), _log(rng, 16, 1500 if fork else 6500)
        case = _pages("", B=B, nodes=rng.randint(1, 64), planes=_log(rng, 1, 32) if fork else 1, ctx_lo=ctx // 3, ctx_hi=ctx,
                      block=block, leaders=rng.randint(1, max(1, B // 2)) if fork else 0, latent=latent, rot=rot, dtype=dtype)
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs --


def _lengths(case):
    """Tokens in the cache and new tokens of each sequence, from the case alone."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["B"])]
    if "nodes" in case:
        new = [case["nodes"]] * case["B"]
    else:
        new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["B"])]
        new[0] = case["new_hi"]
    ctx[0] = case["ctx_hi"]
    return ctx, new


def _latents(shape, C, g, dev, dt):
    """Normalised latent vectors with some strong channels, and rotated shared dimensions behind them."""
    x = torch.empty(shape, dtype=dt, device=dev)
    gain = torch.where(torch.rand(shape[-1], generator=g, device=dev) < 0.04, 2.5, 0.9)
    for part in x.flatten(0, -2).split(1 << 19):
        part.copy_(torch.randn(part.shape, generator=g, device=dev) * gain)
    return x


def _table(need, g, dev, spare, width=None):
    """A pool's size, and each sequence's blocks, scattered over it; -1 behind them."""
    total = sum(need)
    order = torch.randperm(total + spare, generator=g, device=dev).to(torch.int32)
    table = torch.full((len(need), width or max(need)), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at: at + k]
        at += k
    return total + spare, table


def _tree_mask(rng, n):
    """The ancestor mask of a random tree in level order (parent < child)."""
    parent = sorted(rng.randrange(max(1, (i + 2) // 3)) if rng.random() < 0.8 else max(0, i - 1) for i in range(n - 1))
    mask = [[0] * n for _ in range(n)]
    for i in range(n):
        if i:
            mask[i] = list(mask[min(parent[i - 1], i - 1)])
        mask[i][i] = 1
    return mask


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(1000003 * int(seed) + 29)
    rng = random.Random(int(seed))
    ctx, new = _lengths(case)
    bs, C, R, B, dt = case["block"], case["latent"], case["rot"], case["B"], DTYPES[case["dtype"]]
    s = dict(case=case, ctx=ctx, new=new)
    if case["op"] == "pages":
        return _prepare_pages(case, s, g, rng, dev)
    blocks, s["block_table"] = _table([-(-(c + n) // bs) for c, n in zip(ctx, new)], g, dev, 3)
    s["cache_len"] = torch.tensor(ctx, dtype=torch.int32, device=dev)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s["cu_tokens"], T = torch.tensor(starts, dtype=torch.int32, device=dev), starts[-1]
    s["max_tokens"] = max(new)
    if case["op"] == "compact":
        s["cache"] = _latents((case["planes"], blocks, bs, C + R), C, g, dev, dt)
        n, depth = case["nodes"], 8
        path, accept = [], []
        for _ in range(B):  # the chain of first children for a while, then nodes of later levels
            L = rng.randint(0, min(depth, n - 1))
            lead = rng.randint(0, L)
            row = list(range(lead + 1)) + sorted(rng.sample(range(L + 1, n), min(L - lead, n - 1 - L)))
            accept.append(len(row) - 1)
            path.append(row + [-1] * (depth + 1 - len(row)))
        s["path"] = torch.tensor(path, dtype=torch.int32, device=dev)
        s["accept_len"] = torch.tensor(accept, dtype=torch.int32, device=dev)
        return s
    s["cache"] = _latents((blocks, bs, C + R), C, g, dev, dt)
    if case["op"] == "attention":
        s["q"] = (torch.randn(T, case["heads"], C + R, generator=g, device=dev) * 0.8).to(dt)
        s["tree_mask"] = None
        if case["tree"]:
            s["tree_mask"] = torch.tensor([_tree_mask(rng, case["new_hi"]) for _ in new], dtype=torch.uint8, device=dev)
        return s
    # what the two down projections leave: [T, C + R], cut by the call
    s["down"] = (torch.randn(T, C + R, generator=g, device=dev) *
                 torch.where(torch.rand(C + R, generator=g, device=dev) < 0.04, 4.0, 1.5)).to(dt)
    s["norm_weight"] = (1 + 0.2 * torch.randn(C, generator=g, device=dev)).to(dt) if case["norm"] else None
    s["q"] = torch.randn(T, case["heads"], C + R, generator=g, device=dev).to(dt) if case["heads"] else None
    s["inv_freq"] = [500000.0 ** (-2.0 * i / R) for i in range(R // 2)]
    s["inv_freq_dev"] = torch.tensor(s["inv_freq"], dtype=torch.float64, device=dev)
    return s


def _prepare_pages(case, s, g, rng, dev):
    bs, B, leaders = case["block"], case["B"], case["leaders"]
    ctx = s["ctx"]
    width = -(-(max(ctx) + case["nodes"]) // bs) + 1
    if leaders:  # sequence b becomes a fork of one of the first; the others hold nothing yet
        ctx[leaders:] = [0] * (B - leaders)
        s["source"] = [b if b < leaders else b % leaders for b in range(B)]
        keep = [ctx[x] for x in s["source"]]
    else:  # some of the last step's tokens were rejected
        s["source"] = None
        keep = [max(0, c - rng.randint(0, min(8, case["nodes"] - 1))) for c in ctx]
    spare = B * (case["nodes"] // bs + 2) + 5
    held = [-(-c // bs) for c in ctx]
    blocks, table = _table(held, g, dev, spare, width)
    refs = torch.zeros(blocks, dtype=torch.int32, device=dev)
    if not leaders and B > 1:  # every fourth sequence shares the first blocks of the one before it
        for b in range(3, B, 4):
            n = min(held[b], held[b - 1]) - 1
            if n > 0:
                table[b, :n] = table[b - 1, :n]
    refs.index_add_(0, table[table >= 0].long(), torch.ones_like(table[table >= 0]))
    s.update(block_table=table, refs=refs, cache_len=torch.tensor(ctx, dtype=torch.int32, device=dev),
             keep_len=torch.tensor(keep, dtype=torch.int32, device=dev),
             need=torch.full((B,), case["nodes"], dtype=torch.int32, device=dev))
    s["source_dev"] = torch.tensor(s["source"], dtype=torch.int32, device=dev) if leaders else None
    s["cache"] = _latents((case["planes"], blocks, bs, case["latent"] + case["rot"]), case["latent"], g, dev,
                          DTYPES[case["dtype"]])
    return s


# --------------------------------------------------------------- the package --


def _own(s):
    import speculative_decoding_verification_29_gb300 as sv

    op, C = s["case"]["op"], s["case"]["latent"]
    if op == "attention":
        return sv.spec_latent_attention(s["q"], s["cache"], s["block_table"], s["cache_len"], s["cu_tokens"],
                                        max_tokens=s["max_tokens"], value_dim=C, sm_scale=SM_SCALE,
                                        tree_mask=s["tree_mask"])["out"]
    if op == "append":
        q = s["q"][..., C:] if s["q"] is not None else None
        r = sv.spec_latent_append(s["down"][:, :C], s["down"][:, C:], s["cache"], s["block_table"], s["cache_len"],
                                  s["cu_tokens"], inv_freq=s["inv_freq"], interleaved=s["case"]["interleaved"],
                                  norm_weight=s["norm_weight"], eps=1e-6, q_rope=q)
        return [s["cache"]] + ([r["q_out"]] if q is not None else [])
    if op == "compact":
        r = sv.spec_latent_compact(s["cache"], s["block_table"], s["cache_len"], s["accept_len"], s["path"])
        return [s["cache"], r["new_len"]]
    r = sv.spec_pages_update(s["block_table"], s["cache_len"], s["refs"], [s["cache"]], planes=True,
                             keep_len=s["keep_len"], source=s["source_dev"], need=s["need"])
    s["block_table"], s["cache_len"] = r["block_table"], r["cache_len"]  # the loop goes on with these
    return [s["cache"], r["block_table"], r["cache_len"], s["refs"], r["row_status"]]


# ----------------------------------------------------------- the plain forms --


def _sequence_of(s, T):
    """For each packed token: its sequence, and its place among the sequence's new tokens."""
    t = torch.arange(T, device=s["cu_tokens"].device)
    b = torch.searchsorted(s["cu_tokens"], t, right=True, out_int32=True).long() - 1
    return b, t - s["cu_tokens"][b]


def _plain_attention(s):
    q, table, C = s["q"], s["block_table"].long().clamp(min=0), s["case"]["latent"]
    T, H, W = q.shape
    B, n = table.shape[0], s["max_tokens"]
    b, i = _sequence_of(s, T)
    rows = torch.zeros(B, n, H, W, device=q.device)
    rows[b, i] = q.float()
    kv = s["cache"][table].float().view(B, -1, W)
    score = rows.view(B, n * H, W) @ kv.transpose(1, 2)
    score *= SM_SCALE
    slot = torch.arange(score.shape[-1], device=q.device)
    at = slot - s["cache_len"][:, None]  # [B, L]: the slot's place among the new tokens, negative in the context
    new = s["cu_tokens"][1:] - s["cu_tokens"][:-1]
    if s["tree_mask"] is None:
        seen = at[:, None, :] <= torch.arange(n, device=q.device)[:, None]
    else:
        m = s["tree_mask"].bool().gather(2, at.clamp(0, n - 1)[:, None, :].expand(B, n, -1))
        seen = m | (at < 0)[:, None, :]
    seen = seen & (at < new[:, None])[:, None, :]
    score.view(B, n, H, -1).masked_fill_(~seen[:, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    score = score.sub_(torch.where(top > -math.inf, top, torch.zeros_like(top))).exp_()
    total = score.sum(-1, keepdim=True)
    out = (score @ kv[..., :C]) / torch.where(total > 0, total, torch.ones_like(total))
    return out.view(B, n, H, C)[b, i].to(q.dtype)


def _turned(x, pos, s):
    """x [T, heads, R] in fp32, turned by pos * inv_freq (angles in 64 bits)."""
    a = (pos[:, None].double() * s["inv_freq_dev"])[:, None, :]
    c, d = a.cos().float(), a.sin().float()
    x, half = x.float(), c.shape[-1]
    if s["case"]["interleaved"]:
        u, w = x[..., 0::2], x[..., 1::2]
        return torch.stack((u * c - w * d, w * c + u * d), -1).flatten(-2)
    u, w = x[..., :half], x[..., half:]
    return torch.cat((u * c - w * d, w * c + u * d), -1)


def _plain_append(s):
    C, bs, cache = s["case"]["latent"], s["case"]["block"], s["cache"]
    b, i = _sequence_of(s, s["down"].shape[0])
    pos = s["cache_len"][b] + i
    x = s["down"][:, :C].float()
    if s["norm_weight"] is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * s["norm_weight"].float()
    x = torch.cat((x, _turned(s["down"][:, None, C:], pos, s)[:, 0]), -1)
    cache[s["block_table"][b, pos // bs].long(), pos % bs] = x.to(cache.dtype)
    return [cache] + ([_turned(s["q"][..., C:], pos, s).to(cache.dtype)] if s["q"] is not None else [])


def _plain_compact(s):
    bs, cache = s["case"]["block"], s["cache"]
    t = torch.arange(s["path"].shape[1], device=cache.device)
    b, t = torch.nonzero(t <= s["accept_len"][:, None], as_tuple=True)
    src = (s["cache_len"][b] + s["path"][b, t]).long()
    dst = (s["cache_len"][b] + t).long()
    cache[:, s["block_table"][b, dst // bs].long(), dst % bs] = cache[:, s["block_table"][b, src // bs].long(), src % bs]
    return [cache, s["cache_len"] + s["accept_len"] + 1]


def _plain_pages(s):
    bs, old, keep, need, refs = s["case"]["block"], s["block_table"], s["keep_len"], s["need"], s["refs"]
    B, M = old.shape
    j = torch.arange(M, device=old.device)
    kept = (keep + bs - 1) // bs
    table = torch.where(j < kept[:, None], old if s["source_dev"] is None else old[s["source_dev"].long()], -1)
    for t, sign in ((old, -1), (table, 1)):
        refs.scatter_add_(0, t.clamp(min=0).long().flatten(), torch.where(t >= 0, sign, 0).to(torch.int32).flatten())
    last = table.gather(1, (kept - 1).clamp(min=0).long()[:, None])[:, 0]
    writes = (keep % bs > 0) & (need > 0)  # sequences whose next token goes into a block that holds some already
    same = (last[:, None] == last[None, :]) & writes[:, None] & writes[None, :]
    copies = writes & (refs[last.clamp(min=0).long()] - same.tril(-1).sum(1) > 1)  # the last one that shares it keeps it
    more = (keep + need + bs - 1) // bs - kept + copies
    more = torch.where(need > 0, more, torch.zeros_like(more))
    upto = more.cumsum(0)
    free = torch.nonzero(refs == 0)[:, 0].to(torch.int32)
    short = (need > 0) & (upto > free.numel())
    copies = copies & ~short
    first = kept - copies.int()
    at = j - first[:, None]
    takes = (at >= 0) & (at < more[:, None]) & ~short[:, None]
    free = torch.cat((free, free.new_full((1,), -1)))
    new = free[((upto - more)[:, None] + at).clamp(0, free.numel() - 1).long()]
    table = torch.where(takes, new, table)
    refs.scatter_add_(0, last.clamp(min=0).long(), -copies.int())
    refs.scatter_add_(0, table.clamp(min=0).long().flatten(), takes.int().flatten())
    b = torch.nonzero(copies)[:, 0]
    if b.numel():
        s["cache"][:, table[b, (kept - 1)[b].long()].long()] = s["cache"][:, last[b].long()]
    s["block_table"], s["cache_len"] = table, keep.clone()
    return [s["cache"], table, s["cache_len"], refs, torch.where(short, CACHE_BAD, 0).to(torch.int32)]


def run(state):
    if own:
        return _own(state)
    return {"attention": _plain_attention, "append": _plain_append, "compact": _plain_compact,
            "pages": _plain_pages}[state["case"]["op"]](state)


# ------------------------------------------------------------------- figures --


def work(case):
    ctx, new = _lengths(case)
    C, W, bs = case["latent"], case["latent"] + case["rot"], case["block"]
    if case["op"] == "attention":
        H, T = case["heads"], sum(new)
        slots = sum(c + n for c, n in zip(ctx, new))
        pairs = sum(n * c + (n * (n + 1)) // 2 for c, n in zip(ctx, new))
        return {"bytes": 2 * W * slots + 4 * slots // bs + 2 * T * H * (W + C), "flops": 2 * (W + C) * H * pairs}
    if case["op"] == "append":
        return {"bytes": sum(new) * 2 * (2 * W + 2 * case["heads"] * case["rot"]), "flops": 0}
    if case["op"] == "compact":
        return {"bytes": case["B"] * 4.0 * 2 * case["planes"] * W * 2, "flops": 0}  # a path's mean length
    blocks, copies = sum(-(-c // bs) for c in ctx), case["B"] - 1 if case["leaders"] else 0
    return {"bytes": 4 * (3 * blocks + 4 * case["B"]) + 2.0 * copies * case["planes"] * bs * W * 2, "flops": 0}


# ---------------------------------------------------------- the definitions in 64 bits --


def exact(case, seed):
    if case["op"] == "pages":
        return None  # whole numbers and copies
    s = prepare(case, seed)
    return {"attention": _exact_attention, "append": _exact_append, "compact": _exact_compact}[case["op"]](s)


def _exact_attention(s):
    bs, C, start, outs = s["case"]["block"], s["case"]["latent"], 0, []
    for b, (c, n) in enumerate(zip(s["ctx"], s["new"])):
        ids = s["block_table"][b, : -(-(c + n) // bs)].tolist()
        kv = torch.cat([s["cache"][j] for j in ids])[: c + n].double()
        q = s["q"][start: start + n].double()
        start += n
        seen = torch.ones(n, c + n, dtype=torch.bool, device=q.device)
        seen[:, c:] = s["tree_mask"][b, :n, :n].bool() if s["tree_mask"] is not None else seen[:, c:].tril()
        heads = []
        for h in range(q.shape[1]):
            w = (q[:, h] @ kv.T) * SM_SCALE
            heads.append(torch.softmax(w.masked_fill(~seen, -math.inf), -1) @ kv[:, :C])
        outs.append(torch.stack(heads, 1))
    return torch.cat(outs)


def _exact_append(s):
    C, R, bs, start, turned = s["case"]["latent"], s["case"]["rot"], s["case"]["block"], 0, []
    out = s["cache"].double()

    def turn(x, first):
        z = x.double().clone()
        a = torch.arange(first, first + x.shape[0], device=x.device, dtype=torch.float64)
        a = (a[:, None] * s["inv_freq_dev"]).view(x.shape[0], *[1] * (x.dim() - 2), R // 2)
        even, odd = (slice(0, R, 2), slice(1, R, 2)) if s["case"]["interleaved"] else (slice(0, R // 2), slice(R // 2, R))
        pair = torch.complex(z[..., even], z[..., odd]) * torch.polar(torch.ones_like(a), a)
        z[..., even], z[..., odd] = pair.real, pair.imag
        return z

    for b, (c, n) in enumerate(zip(s["ctx"], s["new"])):
        x = s["down"][start: start + n].double()
        if s["q"] is not None:
            turned.append(turn(s["q"][start: start + n, :, C:], c))
        start += n
        y = x[:, :C]
        if s["norm_weight"] is not None:
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / C + 1e-6) * s["norm_weight"].double()
        y = torch.cat((y, turn(x[:, C:], c)), 1)
        for j in range(c // bs, (c + n - 1) // bs + 1):
            lo, hi = max(c, j * bs), min(c + n, (j + 1) * bs)
            out[int(s["block_table"][b, j]), lo - j * bs: hi - j * bs] = y[lo - c: hi - c]
    return [out] + ([torch.cat(turned)] if s["q"] is not None else [])


def _exact_compact(s):
    bs = s["case"]["block"]
    out = s["cache"].double()
    for c, row, L, ids in zip(s["ctx"], s["path"].tolist(), s["accept_len"].tolist(), s["block_table"].tolist()):
        moved = [out[:, ids[(c + p) // bs], (c + p) % bs].clone() for p in row[: L + 1]]
        for t, x in enumerate(moved):
            out[:, ids[(c + t) // bs], (c + t) % bs] = x
    return [out, None]
