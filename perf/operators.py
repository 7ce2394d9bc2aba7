"""Performance cases of the 8-bit paged KV cache: appending rotated keys and values, attention over the cache, and
compaction after tree verification.

The cache of one layer is a pool of blocks. Block i holds `block` tokens of every KV head as e4m3 codes, keys and
values apart, [blocks, kv_heads, block, head_dim], and one power-of-two scale for each block and head, [blocks, kv_heads]
(e8m0). A value is code * scale. `block_table[b]` lists the blocks of sequence b in order; it has `cache_len[b]` tokens in
the cache before the step and the step adds tokens cu_tokens[b] .. cu_tokens[b + 1] - 1 of the packed inputs after them.

`run` computes the operators in elementary torch operations (`own` false) or through the package (`own` true).
"""

import math
import random

import torch

own = False

FP8_MAX = 448.0
SCALE_LO, SCALE_HI = -40, 40  # the scales' exponents
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one user, one token: the latency of a single decode step on a short context
        _attention("attn_decode_one", B=1, new_lo=1, new_hi=1, ctx_lo=517, ctx_hi=517, block=16),
        # a full decode batch on ragged contexts, Llama-3-8B heads
        _attention("attn_decode", B=64, new_lo=1, new_hi=1, ctx_lo=1500, ctx_hi=6500, block=64),
        # a small drafter decoding for the same batch: 64-wide heads, fp16
        _attention("attn_drafter", B=48, new_lo=1, new_hi=1, ctx_lo=900, ctx_hi=3100, block=32, q_heads=16, kv_heads=8,
                   head_dim=64, dtype="fp16"),
        # the target's pass over K = 8 draft tokens and the root, the chain verification batch
        _attention("attn_verify", B=64, new_lo=9, new_hi=9, ctx_lo=1500, ctx_hi=6500, block=64),
        # the target's pass over merged trees of N = 61 nodes
        _attention("attn_tree", B=16, new_lo=61, new_hi=61, ctx_lo=500, ctx_hi=3500, block=32, tree=True),
        # two users with long contexts, K = 8: few rows, a long axis
        _attention("attn_long", B=2, new_lo=9, new_hi=9, ctx_lo=110001, ctx_hi=131072, block=128),
        # prompts of several users after a shared prefix, fp16
        _attention("attn_prompt", B=3, new_lo=1500, new_hi=4096, ctx_lo=1, ctx_hi=1000, block=64, dtype="fp16"),
        # K = 8 draft tokens and the root of one user
        _append("append_one", B=1, new_lo=9, new_hi=9, ctx_lo=517, ctx_hi=517, block=16),
        # the verification batch: queries rotated in the same call
        _append("append_verify", B=64, new_lo=9, new_hi=9, ctx_lo=1500, ctx_hi=6500, block=64, q_heads=32),
        # prompts, ragged, interleaved pairs over half of the head
        _append("append_prompt", B=8, new_lo=1500, new_hi=4096, ctx_lo=0, ctx_hi=1000, block=64, interleaved=True, rot=64,
                dtype="fp16"),
        # accepted tree paths of one user, one layer
        _compact("compact_one", B=1, nodes=61, planes=1, ctx_lo=517, ctx_hi=517, block=16),
        # accepted tree paths of the tree batch in every one of 32 layers
        _compact("compact_tree", B=16, nodes=61, planes=32, ctx_lo=180, ctx_hi=420, block=64),
    ]


def _attention(name, *, B, new_lo, new_hi, ctx_lo, ctx_hi, block, q_heads=32, kv_heads=8, head_dim=128, dtype="bf16",
               tree=False):
    return dict(name=name, op="attention", B=B, new_lo=new_lo, new_hi=new_hi, ctx_lo=ctx_lo, ctx_hi=ctx_hi, block=block,
                q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, dtype=dtype, tree=tree)


def _append(name, *, B, new_lo, new_hi, ctx_lo, ctx_hi, block, q_heads=0, kv_heads=8, head_dim=128, dtype="bf16", rot=None,
            interleaved=False):
    return dict(name=name, op="append", B=B, new_lo=new_lo, new_hi=new_hi, ctx_lo=ctx_lo, ctx_hi=ctx_hi, block=block,
                q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, dtype=dtype, rot=head_dim if rot is None else rot,
                interleaved=interleaved)


def _compact(name, *, B, nodes, planes, ctx_lo, ctx_hi, block, kv_heads=8, head_dim=128):
    return dict(name=name, op="compact", B=B, nodes=nodes, planes=planes, ctx_lo=ctx_lo, ctx_hi=ctx_hi, block=block,
                kv_heads=kv_heads, head_dim=head_dim)


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the listed ones' ranges: decode, verification, tree, long and prompt attention, appends, compactions."""
    op = rng.choice(["attention"] * 4 + ["append"] * 2 + ["compact"])
    block = rng.choice([16, 32, 64, 128])
    head_dim = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    if op == "attention":
        kind = rng.choice(["decode", "verify", "verify", "tree", "long", "prompt"])
        group = rng.choice([1, 2, 3, 4, 7, 8])
        B, new = _log(rng, 1, 64), (1, 1)
        ctx = _log(rng, 16, 6500)
        if kind == "verify":
            K1 = rng.randint(2, 17)
            new = (rng.randint(1, K1), K1)
        elif kind == "tree":
            B, new = _log(rng, 1, 16), (rng.randint(5, 64),) * 2
            ctx = _log(rng, 16, 3500)
        elif kind == "long":
            B, new, ctx = rng.randint(1, 2), (1, rng.randint(1, 9)), _log(rng, 20000, 131072)
        elif kind == "prompt":
            top = _log(rng, 65, 4096)
            B, new, ctx = rng.randint(1, 3), (top // 2, top), _log(rng, 1, 1000)
        return {k: v for k, v in _attention(
            "", B=B, new_lo=new[0], new_hi=new[1], ctx_lo=ctx // 3, ctx_hi=ctx, block=block, q_heads=group * kv_heads if
            group * kv_heads <= 32 else kv_heads * (32 // kv_heads), kv_heads=kv_heads, head_dim=head_dim,
            dtype=rng.choice(["bf16", "fp16"]), tree=kind == "tree").items() if k != "name"}
    if op == "append":
        prompt = rng.random() < 0.4
        top = _log(rng, 65, 4096) if prompt else rng.randint(1, 61)
        B = rng.randint(1, 8) if prompt else _log(rng, 1, 64)
        ctx = _log(rng, 1, 6500)
        return {k: v for k, v in _append(
            "", B=B, new_lo=max(1, top // 2), new_hi=top, ctx_lo=ctx // 3, ctx_hi=ctx, block=block,
            q_heads=rng.choice([0, 1, 4]) * kv_heads, kv_heads=kv_heads, head_dim=head_dim,
            dtype=rng.choice(["bf16", "fp16", "fp32"]), rot=rng.choice([head_dim, head_dim // 2, 32]),
            interleaved=rng.random() < 0.3).items() if k != "name"}
    ctx = _log(rng, 16, 420)
    return {k: v for k, v in _compact("", B=_log(rng, 1, 16), nodes=rng.randint(9, 64), planes=_log(rng, 1, 32),
                                      ctx_lo=ctx // 3, ctx_hi=ctx, block=block, kv_heads=kv_heads,
                                      head_dim=head_dim).items() if k != "name"}


# ------------------------------------------------------------------ inputs --


def _lengths(case):
    """Tokens in the cache and new tokens of each sequence, from the case alone."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["B"])]
    if case["op"] == "compact":
        return ctx, [case["nodes"]] * case["B"]
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["B"])]
    ctx[0], new[0] = case["ctx_hi"], case["new_hi"]
    return ctx, new


def _need(amax):
    """The exponent of the least scale that holds `amax` (448 codes up): amax = m 2^x, 0.5 <= m < 1, 448 = 0.875 2^9."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8)
    return torch.where(amax > 0, e, torch.full_like(e, SCALE_LO)).clamp(SCALE_LO, SCALE_HI)


def _codes(x, e):
    """Codes of x (fp32) under the exponents e: round to nearest even, clamped to +-448."""
    return torch.ldexp(x, -e).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)


def _pool(case, g, blocks, dev):
    """A pool of filled blocks: codes [blocks, H, block, D] and scales [blocks, H], keys with some strong channels."""
    H, D, bs = case["kv_heads"], case["head_dim"], case["block"]
    out = []
    for spread in (3.0, 1.0):
        x = torch.randn(blocks, H, bs, D, generator=g, device=dev)
        x *= torch.where(torch.rand(1, H, 1, D, generator=g, device=dev) < 0.04, spread, 0.8)
        x *= torch.exp2(torch.randn(blocks, 1, 1, 1, generator=g, device=dev) * 0.3)
        e = _need(x.abs().amax((2, 3)))
        out += [_codes(x, e[:, :, None, None]).view(torch.uint8), (e + 127).to(torch.uint8)]
    return out  # k, k scale, v, v scale


def _tables(ctx, new, bs, g, dev):
    """A pool's size, and each sequence's blocks, scattered over it; -1 behind them."""
    need = [-(-(c + n) // bs) for c, n in zip(ctx, new)]
    total = sum(need)
    order = torch.randperm(total + 3, generator=g, device=dev).to(torch.int32)
    table = torch.full((len(ctx), max(need)), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at: at + k]
        at += k
    return total + 3, table


def _tree(rng, n):
    """Parents of a random tree in level order (parent < child), its depths and its ancestor mask."""
    parent = sorted(rng.randrange(max(1, (i + 2) // 3)) if rng.random() < 0.8 else max(0, i - 1) for i in range(n - 1))
    parent = [0] + [min(p, i) for i, p in enumerate(parent)]
    mask = [[0] * n for _ in range(n)]
    depth = [0] * n
    for i in range(n):
        if i:
            mask[i] = list(mask[parent[i]])
            depth[i] = depth[parent[i]] + 1
        mask[i][i] = 1
    return parent, depth, mask


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(1000003 * int(seed) + 17)
    rng = random.Random(int(seed))
    ctx, new = _lengths(case)
    bs, H, D = case["block"], case["kv_heads"], case["head_dim"]
    s = dict(case=case, ctx=ctx, new=new, max_tokens=max(new), max_len=max(c + n for c, n in zip(ctx, new)))
    blocks, s["block_table"] = _tables(ctx, new, bs, g, dev)
    s["cache_len"] = torch.tensor(ctx, dtype=torch.int32, device=dev)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s["cu_tokens"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    T = starts[-1]
    if case["op"] == "compact":
        P = case["planes"]
        k, ks, v, vs = _pool(dict(case, kv_heads=P * H), g, blocks, dev)
        for name, x in (("k_cache", k), ("v_cache", v)):
            s[name] = x.view(blocks, P, H, bs, D).transpose(0, 1).contiguous()
        for name, x in (("k_scale", ks), ("v_scale", vs)):
            s[name] = x.view(blocks, P, H).transpose(0, 1).contiguous()
        n, depth = case["nodes"], 8
        path, accept = [], []
        for _ in range(case["B"]):  # the chain of first children for a while, then nodes of later levels
            L = rng.randint(0, min(depth, n - 1))
            lead = rng.randint(0, L)
            tail = sorted(rng.sample(range(L + 1, n), min(L - lead, n - 1 - L)))
            row = list(range(lead + 1)) + tail
            accept.append(len(row) - 1)
            path.append(row + [-1] * (depth + 1 - len(row)))
        s["path"] = torch.tensor(path, dtype=torch.int32, device=dev)
        s["accept_len"] = torch.tensor(accept, dtype=torch.int32, device=dev)
        s["path_host"], s["accept_host"] = path, accept
        return s
    s["k_cache"], s["k_scale"], s["v_cache"], s["v_scale"] = _pool(case, g, blocks, dev)
    dt = DTYPES[case["dtype"]]
    if case["op"] == "attention":
        s["q"] = (torch.randn(T, case["q_heads"], D, generator=g, device=dev) * 1.3).to(dt)
        s["sm_scale"] = D ** -0.5
        s["tree_mask"] = None
        if case["tree"]:
            s["tree_mask"] = torch.tensor([_tree(rng, case["new_hi"])[2] for _ in new], dtype=torch.uint8, device=dev)
        return s
    s["k"] = (torch.randn(T, H, D, generator=g, device=dev) *
              torch.where(torch.rand(1, H, D, generator=g, device=dev) < 0.04, 3.0, 0.8)).to(dt)
    s["v"] = (torch.randn(T, H, D, generator=g, device=dev) * 0.8).to(dt)
    s["q"] = torch.randn(T, case["q_heads"], D, generator=g, device=dev).to(dt) if case["q_heads"] else None
    s["inv_freq"] = [500000.0 ** (-2.0 * i / case["rot"]) for i in range(case["rot"] // 2)]
    s["inv_freq_dev"] = torch.tensor(s["inv_freq"], dtype=torch.float64, device=dev)
    s["interleaved"] = case["interleaved"]
    return s


# --------------------------------------------------------------- the package --


def _own(s):
    import speculative_decoding_verification_29_gb300 as sv

    op = s["case"]["op"]
    cache = (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["block_table"], s["cache_len"])
    if op == "attention":
        return sv.spec_kv8_attention(s["q"], *cache, s["cu_tokens"], max_tokens=s["max_tokens"], sm_scale=s["sm_scale"],
                                     tree_mask=s["tree_mask"])["out"]
    if op == "append":
        r = sv.spec_kv8_append(s["k"], s["v"], *cache, s["cu_tokens"], inv_freq=s["inv_freq"],
                               interleaved=s["interleaved"], q=s["q"])
        return _cache(s, q=r.get("q_out"))
    r = sv.spec_kv8_compact(*cache, s["accept_len"], s["path"])
    return _cache(s, new_len=r["new_len"])


def _cache(s, **more):
    """The cache as the values its bytes stand for: e4m3 codes and e8m0 scales."""
    out = {k: s[k].view(torch.float8_e4m3fn) for k in ("k_cache", "v_cache")}
    out.update({k: s[k].view(torch.float8_e8m0fnu) for k in ("k_scale", "v_scale")})
    out.update({k: v for k, v in more.items() if v is not None})
    return out


# ----------------------------------------------------------- the plain forms --


def _sequence_of(s, T):
    """For each packed token: its sequence, and its place among the sequence's new tokens."""
    t = torch.arange(T, device=s["cu_tokens"].device)
    b = torch.searchsorted(s["cu_tokens"], t, right=True, out_int32=True).long() - 1
    return b, t - s["cu_tokens"][b]


def _gathered(codes, scales, table):
    """fp32 values of the blocks of `table` [B, n]: [B, H, n * block, D]."""
    B, n = table.shape
    x = codes.view(torch.float8_e4m3fn)[table].float()
    x = torch.ldexp(x, (scales[table].int() - 127)[..., None, None])
    return x.transpose(1, 2).reshape(B, x.shape[2], n * x.shape[3], x.shape[4])


def _plain_attention(s):
    q, table = s["q"], s["block_table"].long().clamp(min=0)
    T, Hq, D = q.shape
    H, B, n = s["k_cache"].shape[1], table.shape[0], s["max_tokens"]
    g = Hq // H
    b, i = _sequence_of(s, T)
    rows = torch.zeros(B, n, Hq, D, device=q.device)
    rows[b, i] = q.float()
    rows = rows.view(B, n, H, g, D).permute(0, 2, 1, 3, 4).reshape(B, H, n * g, D)
    score = rows @ _gathered(s["k_cache"], s["k_scale"], table).transpose(2, 3)
    score *= s["sm_scale"]
    slot = torch.arange(score.shape[-1], device=q.device)
    at = slot - s["cache_len"][:, None]  # [B, L]: the slot's place among the new tokens, negative in the context
    new = s["cu_tokens"][1:] - s["cu_tokens"][:-1]
    if s["tree_mask"] is None:
        seen = at[:, None, :] <= torch.arange(n, device=q.device)[:, None]
    else:
        m = s["tree_mask"].bool().gather(2, at.clamp(0, n - 1)[:, None, :].expand(B, n, -1))
        seen = m | (at < 0)[:, None, :]
    seen = seen & (at < new[:, None])[:, None, :]
    score.view(B, H, n, g, -1).masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    score = score.sub_(torch.where(top > -math.inf, top, torch.zeros_like(top))).exp_()
    total = score.sum(-1, keepdim=True)
    v = _gathered(s["v_cache"], s["v_scale"], table)
    v = v.masked_fill_((at >= new[:, None])[:, None, :, None], 0.0)
    out = (score @ v) / torch.where(total > 0, total, torch.ones_like(total))
    out = out.view(B, H, n, g, D).permute(0, 2, 1, 3, 4).reshape(B, n, Hq, D)
    return out[b, i].to(q.dtype)


def _turned(x, pos, s):
    """x [T, H, D] in fp32, its first `rot` dimensions turned by pos * inv_freq (angles in 64 bits)."""
    f = s["inv_freq_dev"]
    a = pos[:, None].double() * f
    c, d = a.cos().float()[:, None, :], a.sin().float()[:, None, :]
    x, half = x.float(), f.numel()
    r = x[..., : 2 * half]
    u, w = (r[..., 0::2], r[..., 1::2]) if s["interleaved"] else (r[..., :half], r[..., half:])
    u, w = u * c - w * d, w * c + u * d
    r = torch.stack((u, w), -1).flatten(-2) if s["interleaved"] else torch.cat((u, w), -1)
    return torch.cat((r, x[..., 2 * half:]), -1)


def _plain_append(s):
    T, H, D = s["k"].shape
    bs = s["k_cache"].shape[2]
    b, i = _sequence_of(s, T)
    slot = s["cache_len"][b] + i
    block = s["block_table"][b, slot // bs].long()
    first = s["block_table"].gather(1, (s["cache_len"] // bs).long()[:, None].clamp(max=s["block_table"].shape[1] - 1))
    kept = (s["cache_len"] % bs) > 0  # sequences whose first block already holds tokens
    first = first[:, 0].long()
    for x, codes, scales in ((_turned(s["k"], slot, s), s["k_cache"], s["k_scale"]),
                             (s["v"].float(), s["v_cache"], s["v_scale"])):
        old = scales.int() - 127
        e = torch.full_like(old, -1000)
        e.scatter_reduce_(0, block[:, None].expand(T, H), _need(x.abs().amax(-1)), "amax")
        e[first[kept]] = torch.maximum(e[first[kept]], old[first[kept]])
        e = torch.where(e > -1000, e, old)
        grown = first[kept]
        codes[grown] = _codes(torch.ldexp(codes[grown].view(torch.float8_e4m3fn).float(), old[grown][..., None, None]),
                              e[grown][..., None, None]).view(torch.uint8)
        codes[block, :, slot % bs] = _codes(x, e[block][..., None]).view(torch.uint8)
        scales.copy_(e + 127)
    return _cache(s, q=None if s["q"] is None else _turned(s["q"], slot, s).to(s["q"].dtype))


def _plain_compact(s):
    B, D1 = s["path"].shape
    P, _, H, bs, D = s["k_cache"].shape
    t = torch.arange(D1, device=s["path"].device)
    b, t = torch.nonzero(t <= s["accept_len"][:, None], as_tuple=True)
    src = (s["cache_len"][b] + s["path"][b, t]).long()
    dst = (s["cache_len"][b] + t).long()
    from_, to = s["block_table"][b, src // bs].long(), s["block_table"][b, dst // bs].long()
    for codes, scales in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])):
        old = scales.int() - 127  # [P, blocks, H]
        x = codes[:, from_, :, src % bs].view(torch.float8_e4m3fn).float()  # [M, P, H, D]
        x = torch.ldexp(x, old[:, from_].transpose(0, 1)[..., None])
        e = old.scatter_reduce(1, to[None, :, None].expand(P, -1, H), _need(x.abs().amax(-1)).transpose(0, 1), "amax")
        held = codes[:, to].view(torch.float8_e4m3fn).float()  # a destination block keeps its values when its scale grows
        codes[:, to] = _codes(torch.ldexp(held, (old[:, to])[..., None, None]), e[:, to][..., None, None]).view(torch.uint8)
        codes[:, to, :, dst % bs] = _codes(x, e[:, to].transpose(0, 1)[..., None]).view(torch.uint8)
        scales.copy_(e + 127)
    return _cache(s, new_len=s["cache_len"] + s["accept_len"] + 1)


def run(state):
    if own:
        return _own(state)
    return {"attention": _plain_attention, "append": _plain_append, "compact": _plain_compact}[state["case"]["op"]](state)


# ------------------------------------------------------------------- figures --


def work(case):
    ctx, new = _lengths(case)
    H, D = case["kv_heads"], case["head_dim"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}.get(case.get("dtype"), 0)
    bs = case["block"]
    if case["op"] == "attention":
        Hq, T = case["q_heads"], sum(new)
        blocks = sum(-(-(c + n) // bs) for c, n in zip(ctx, new))
        pairs = sum(n * c + (n * (n + 1)) // 2 for c, n in zip(ctx, new))
        return {"bytes": 2 * H * D * sum(c + n for c, n in zip(ctx, new)) + 2 * H * blocks + 4 * blocks + 2 * T * Hq * D * size,
                "flops": 4 * D * Hq * pairs}
    if case["op"] == "append":
        T = sum(new)
        return {"bytes": T * (2 * H * D * (size + 1) + 2 * case["q_heads"] * D * size), "flops": 0}
    moved = case["B"] * 4.0  # a path's mean length
    return {"bytes": moved * 2 * case["planes"] * H * D * 2, "flops": 0}


# ---------------------------------------------------------- the definitions in 64 bits --


def exact(case, seed):
    s = prepare(case, seed)
    return {"attention": _exact_attention, "append": _exact_append, "compact": _exact_compact}[case["op"]](s)


def _value64(codes, scales):
    """code * scale of one block [H, block, D] in 64 bits."""
    return codes.view(torch.float8_e4m3fn).double() * (2.0 ** (scales.double() - 127))[:, None, None]


def _exact_attention(s):
    bs, start, outs = s["case"]["block"], 0, []
    for b, (c, n) in enumerate(zip(s["ctx"], s["new"])):
        ids = s["block_table"][b, : -(-(c + n) // bs)].tolist()
        k, v = (torch.cat([_value64(s[x + "_cache"][j], s[x + "_scale"][j]) for j in ids], 1)[:, : c + n] for x in "kv")
        q = s["q"][start: start + n].double()
        start += n
        seen = torch.ones(n, c + n, dtype=torch.bool, device=q.device)
        seen[:, c:] = s["tree_mask"][b, :n, :n].bool() if s["tree_mask"] is not None else seen[:, c:].tril()
        g = q.shape[1] // k.shape[0]
        heads = []
        for h in range(q.shape[1]):
            w = (q[:, h] @ k[h // g].T) * s["sm_scale"]
            heads.append(torch.softmax(w.masked_fill(~seen, -math.inf), -1) @ v[h // g])
        outs.append(torch.stack(heads, 1))
    return torch.cat(outs)


def _exponent(x):
    """The least e in range with max|x| <= 448 * 2^e, for each head of x [H, ...]."""
    top = x.abs().flatten(1).amax(1).tolist()
    out = []
    for a in top:
        e = SCALE_LO
        while e < SCALE_HI and a > FP8_MAX * 2.0 ** e:
            e += 1
        out.append(e)
    return torch.tensor(out, dtype=torch.float64, device=x.device)


def _exact_append(s):
    """Codes are given as value / scale, before their rounding."""
    bs, start, turned = s["case"]["block"], 0, []
    rot, f = s["case"]["rot"], s["inv_freq_dev"]
    out = {x: s[x].view(torch.float8_e4m3fn).double() for x in ("k_cache", "v_cache")}
    out.update({x: 2.0 ** (s[x].double() - 127) for x in ("k_scale", "v_scale")})

    def turn(x, first):
        z = x.double().clone()
        r = x.double()[..., :rot]
        a = torch.arange(first, first + x.shape[0], device=x.device, dtype=torch.float64)[:, None, None] * f
        even, odd = (slice(0, rot, 2), slice(1, rot, 2)) if s["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
        pair = torch.complex(r[..., even], r[..., odd]) * torch.polar(torch.ones_like(a), a)
        z[..., even], z[..., odd] = pair.real, pair.imag
        return z

    for b, (c, n) in enumerate(zip(s["ctx"], s["new"])):
        tok = slice(start, start + n)
        start += n
        if s["q"] is not None:
            turned.append(turn(s["q"][tok], c))
        for name, x in (("k", turn(s["k"][tok], c)), ("v", s["v"][tok].double())):
            codes, scales = out[name + "_cache"], out[name + "_scale"]
            for j in range(c // bs, (c + n - 1) // bs + 1):
                lo, hi = max(c, j * bs), min(c + n, (j + 1) * bs)
                block = int(s["block_table"][b, j])
                part = x[lo - c: hi - c].transpose(0, 1)
                scale = 2.0 ** _exponent(part)
                if lo > j * bs:
                    scale = torch.maximum(scale, scales[block])
                    codes[block] = codes[block] * (scales[block] / scale)[:, None, None]
                codes[block, :, lo - j * bs: hi - j * bs] = part / scale[:, None, None]
                scales[block] = scale
    if s["q"] is not None:
        out["q"] = torch.cat(turned)
    return out


def _exact_compact(s):
    bs = s["case"]["block"]
    out = {x: s[x].view(torch.float8_e4m3fn).double() for x in ("k_cache", "v_cache")}
    out.update({x: 2.0 ** (s[x].double() - 127) for x in ("k_scale", "v_scale")})
    for codes, scales in ((out["k_cache"], out["k_scale"]), (out["v_cache"], out["v_scale"])):
        for b, c in enumerate(s["ctx"]):
            row = s["path_host"][b][: s["accept_host"][b] + 1]
            at = [(int(s["block_table"][b, (c + p) // bs]), (c + p) % bs) for p in row]
            x = [(codes[:, k, :, o] * scales[:, k, :, None]).clone() for k, o in at]  # [P, H, D] each
            for t, z in enumerate(x):
                block, slot = int(s["block_table"][b, (c + t) // bs]), (c + t) % bs
                scale = 2.0 ** _exponent(z.flatten(0, 1)).view(z.shape[:2])
                scale = torch.maximum(scale, scales[:, block])
                codes[:, block] = codes[:, block] * (scales[:, block] / scale)[..., None, None]
                scales[:, block] = scale
                codes[:, block, :, slot] = z / scale[..., None]
    out["new_len"] = None
    return out
