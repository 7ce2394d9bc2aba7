"""Plain 64-bit forms of the 8-bit paged KV cache's operators, on the CPU, one
sequence, block and head at a time, and the inputs of their tests. Shares no
code with the library."""

from __future__ import annotations

import math
import random

import torch

EXP_LO, EXP_HI, CODE_MAX = -40, 40, 448.0
TILE = 128  # slots over which softmax weights share a power of two


def need(amax: float) -> int:
    """Least e in range with amax <= 448 * 2^e."""
    e = EXP_LO
    while e < EXP_HI and amax > CODE_MAX * 2.0 ** e:
        e += 1
    return e


def finite_amax(x: torch.Tensor) -> float:
    f = x[torch.isfinite(x)]
    return float(f.abs().max()) if f.numel() else 0.0


def to_codes(x: torch.Tensor, e: int) -> torch.Tensor:
    """uint8 codes of x (fp64) at scale 2^e; NaN and infinities give the NaN code 0x7f."""
    y = (x * 2.0 ** -e).clamp(-CODE_MAX, CODE_MAX).float().to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.where(torch.isfinite(x), y, torch.full_like(y, 0x7F))


def to_values(codes: torch.Tensor, byte: int) -> torch.Tensor:
    e = min(max(int(byte) - 127, EXP_LO), EXP_HI)
    return codes.view(torch.float8_e4m3fn).double() * 2.0 ** e


def rotate(x, pos, inv_freq, interleaved):
    """x [H, D] fp64 turned to position pos."""
    if inv_freq is None:
        return x
    x = x.clone()
    r = 2 * len(inv_freq)
    for i, f in enumerate(inv_freq):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
        c, s = math.cos(pos * f), math.sin(pos * f)
        u, w = x[:, a].clone(), x[:, b].clone()
        x[:, a], x[:, b] = u * c - w * s, w * c + u * s
    return x


class Cache:
    """A pool with scattered blocks, on the CPU; to(dev) gives the call's arguments."""

    def __init__(self, ctx, new, H, D, bs, seed=0, extra_blocks=3, layout="hnd", stale=0xFF):
        g = torch.Generator().manual_seed(seed)
        self.ctx, self.new, self.H, self.D, self.bs = list(ctx), list(new), H, D, bs
        need_b = [-(-(c + n) // bs) for c, n in zip(ctx, new)]
        self.num = sum(need_b) + extra_blocks
        order = torch.randperm(self.num, generator=g).to(torch.int32)
        self.table = torch.full((len(ctx), max(max(need_b), 1) + 1), -7, dtype=torch.int32)
        at = 0
        for b, k in enumerate(need_b):
            self.table[b, :k] = order[at: at + k]
            at += k
        self.layout = layout
        shape = (self.num, H, bs, D)
        self.k, self.v = torch.full(shape, stale, dtype=torch.uint8), torch.full(shape, stale, dtype=torch.uint8)
        self.ks, self.vs = (torch.randint(100, 140, (self.num, H), generator=g, dtype=torch.uint8) for _ in range(2))
        self.len = torch.tensor(ctx, dtype=torch.int32)
        self.cu = torch.tensor([0] + list(torch.tensor(list(new)).cumsum(0)), dtype=torch.int32)
        self.g = g

    def fill(self, upto=None, spread=1.0):
        """Random entries at positions 0 .. upto[b] - 1 (context and new tokens when None)."""
        for b, (c, n) in enumerate(zip(self.ctx, self.new)):
            end = c + n if upto is None else upto[b]
            for j in range(-(-end // self.bs)):
                cnt = min(self.bs, end - j * self.bs)
                i = int(self.table[b, j])
                for codes, scales in ((self.k, self.ks), (self.v, self.vs)):
                    for h in range(self.H):
                        x = torch.randn(cnt, self.D, generator=self.g, dtype=torch.float64) * \
                            2.0 ** float(torch.randn(1, generator=self.g) * spread)
                        e = need(float(x.abs().max()))
                        codes[i, h, :cnt], scales[i, h] = to_codes(x, e), e + 127
        return self

    def entry(self, codes, scales, b, t):
        """[H, D] values at position t."""
        i, s = int(self.table[b, t // self.bs]), t % self.bs
        return torch.stack([to_values(codes[i, h, s], scales[i, h]) for h in range(self.H)])

    def rows(self, codes, scales, b, end):
        """[H, end, D] values of positions 0 .. end - 1, and their codes and exponents."""
        vals, raw, exps = [], [], []
        for j in range(-(-end // self.bs)):
            i = int(self.table[b, j])
            e = scales[i].int().sub(127).clamp(EXP_LO, EXP_HI)
            c = codes[i].view(torch.float8_e4m3fn).double()
            raw.append(c)
            vals.append(c * torch.pow(2.0, e.double())[:, None, None])
            exps.append(e.double()[:, None].expand(self.H, self.bs))
        return tuple(torch.cat(x, 1)[:, :end] for x in (vals, raw, exps))

    def to(self, dev):
        def place(x):
            if self.layout == "nhd":  # slots outside heads
                return x.transpose(1, 2).contiguous().to(dev).transpose(1, 2)
            if self.layout == "padded":
                y = torch.full((self.num + 1, self.H + 1, self.bs + 2, self.D + 32), 0x7F, dtype=torch.uint8, device=dev)
                y[: self.num, : self.H, : self.bs, : self.D] = x.to(dev)
                return y[: self.num, : self.H, : self.bs, : self.D]
            return x.clone().to(dev)

        return [place(self.k), place(self.v), self.ks.clone().to(dev), self.vs.clone().to(dev), self.table.to(dev),
                self.len.to(dev)]


def append(c: Cache, k, v, inv_freq=None, interleaved=False, positions=None):
    """The cache's arrays after the call, in 64 bits: codes, scales, and the values before their rounding
    (NaN where a slot is not written)."""
    out = [x.clone() for x in (c.k, c.v, c.ks, c.vs)]
    raw = [torch.full(c.k.shape, math.nan, dtype=torch.float64) for _ in range(2)]
    for b, (ctx, n) in enumerate(zip(c.ctx, c.new)):
        t0 = int(c.cu[b])
        for j in range(ctx // c.bs, -(-(ctx + n) // c.bs) if n else 0):
            i, base = int(c.table[b, j]), j * c.bs
            lo, hi = max(ctx, base), min(ctx + n, base + c.bs)
            for which, x in enumerate((k, v)):
                codes, scales = out[which], out[2 + which]
                part = []
                for p in range(lo, hi):
                    t = t0 + p - ctx
                    z = x[t].double()
                    if which == 0:
                        z = rotate(z, int(positions[t]) if positions is not None else p, inv_freq, interleaved)
                    part.append(z)
                part = torch.stack(part, 1)  # [H, cnt, D]
                for h in range(c.H):
                    e = need(finite_amax(part[h].float().double()))
                    if lo > base:
                        old = min(max(int(scales[i, h]) - 127, EXP_LO), EXP_HI)
                        e = max(e, old)
                        if e > old:
                            keep = to_codes(codes[i, h].view(torch.float8_e4m3fn).double() * 2.0 ** old, e)
                            codes[i, h] = keep
                    codes[i, h, lo - base: hi - base] = to_codes(part[h], e)
                    raw[which][i, h, lo - base: hi - base] = part[h]
                    scales[i, h] = e + 127
    return out, raw


def compact(c: Cache, path, accept):
    out = [x.clone() for x in (c.k, c.v, c.ks, c.vs)]
    for b, ctx in enumerate(c.ctx):
        L = int(accept[b])
        for codes, scales, src_c, src_s in ((out[0], out[2], c.k, c.ks), (out[1], out[3], c.v, c.vs)):
            x = [c.entry(src_c, src_s, b, ctx + int(path[b][t])) for t in range(L + 1)]
            for j in range(ctx // c.bs, (ctx + L) // c.bs + 1):
                i = int(c.table[b, j])
                ts = [t for t in range(L + 1) if (ctx + t) // c.bs == j]
                for h in range(c.H):
                    old = min(max(int(src_s[i, h]) - 127, EXP_LO), EXP_HI)
                    e = max([old] + [need(finite_amax(x[t][h])) for t in ts])
                    if e > old:
                        codes[i, h] = to_codes(src_c[i, h].view(torch.float8_e4m3fn).double() * 2.0 ** old, e)
                        scales[i, h] = e + 127
                    for t in ts:
                        if int(path[b][t]) != t or e > old:
                            codes[i, h, (ctx + t) % c.bs] = to_codes(x[t][h], e)
    return out


def attention(c: Cache, q, scale, tree=None):
    """(out, tolerance) [T, Hq, D] in 64 bits for q's type.

    Tolerance, per element, with A = sum_t p_t |v_t|: half a step of the output's type on the result; the weights'
    rounding, two e4m3 terms for bf16 (2^-4 of 2^-4, on weights whose share of the tile's largest is at least the
    second term's reach) and three for fp16 (bounded by fp16 rounding of the weight, 2^-11, and 2^-4 of 2^-8), relative
    to A; the codes' floor, half of e4m3's least step 2^-9 where the tile's largest weight is between 2^7 and 2^8, so
    2^-10 / 2^7 = 2^-17 of that weight for every slot; and the scores' error ds: the queries' terms (4 bits and a sign
    each: 8 bits in two, 11 in three) are exact down to a floor of 2^-17 of the largest query element, the products' sums
    and the exponent's rounding take 2^-20 of sum |q k|, and ds moves the weights by 2 ds relative to A."""
    bf = q.dtype == torch.bfloat16
    half, wrel = (2.0 ** -8, 2.0 ** -8) if bf else (2.0 ** -11, 2.0 ** -11)
    T, Hq, D = q.shape
    g = Hq // c.H
    out, tol = torch.full((T, Hq, D), math.nan, dtype=torch.float64), torch.zeros(T, Hq, D, dtype=torch.float64)
    for b, (ctx, n) in enumerate(zip(c.ctx, c.new)):
        if not n:
            continue
        t0 = int(c.cu[b])
        k, _, _ = c.rows(c.k, c.ks, b, ctx + n)
        v, vraw, vexp = c.rows(c.v, c.vs, b, ctx + n)
        seen = torch.ones(n, ctx + n, dtype=torch.bool)
        seen[:, ctx:] = tree[b, :n, :n].bool() if tree is not None else torch.ones(n, n).tril().bool()
        qb = q[t0: t0 + n].double()
        qmax = float(qb[torch.isfinite(qb)].abs().max())
        for a in range(Hq):
            h = a // g
            for i in range(n):
                s = seen[i]
                if not s.any():
                    out[t0 + i, a] = 0.0
                    continue
                kk, vv = k[h][s], v[h][s]
                w = (kk @ qb[i, a]) * scale
                p = torch.softmax(w, 0)
                o = p @ vv
                A = p @ vv.abs()
                ds = (abs(scale) * (kk.abs().sum(-1) * qmax * 2.0 ** -17 + (kk.abs() @ qb[i, a].abs()) * 2.0 ** -20)).max()
                pos = torch.nonzero(s)[:, 0]
                wt = p * torch.pow(2.0, vexp[h][s])
                floor = torch.zeros(D, dtype=torch.float64)
                for tile in range(0, ctx + n, TILE):
                    m = (pos >= tile) & (pos < tile + TILE)
                    if m.any():
                        floor += wt[m].max() * 2.0 ** -17 * vraw[h][s][m].abs().sum(0)
                out[t0 + i, a] = o
                tol[t0 + i, a] = o.abs() * half * 1.01 + A * (wrel + 2 * ds + 2.0 ** -20) + floor + 1e-30
                if not bf:
                    tol[t0 + i, a] += 2.0 ** -25  # fp16's least step, halved
    return out, tol


def tree_mask(rng: random.Random, B, N):
    """Self-inclusive ancestor masks of random trees, and depths."""
    mask, depth = torch.zeros(B, N, N, dtype=torch.uint8), torch.zeros(B, N, dtype=torch.int32)
    for b in range(B):
        for i in range(N):
            if i:
                p = rng.randrange(max(0, i - 5), i)
                mask[b, i] = mask[b, p]
                depth[b, i] = depth[b, p] + 1
            mask[b, i, i] = 1
    return mask, depth
