"""Plain 64-bit forms of the paged latent cache's operators and of the pages, on the CPU, one sequence at a time, the inputs
of their tests, and the tolerances' derivation. Shares no code with the library."""

from __future__ import annotations

import math

import torch


def half_step(dt):
    return torch.finfo(dt).eps / 2


class Cache:
    """A pool with scattered blocks, on the CPU; to(dev) gives the calls' arguments. What no sequence holds is NaN."""

    def __init__(self, ctx, new, C, R, bs, dt, seed=0, layout="dense"):
        g = torch.Generator().manual_seed(seed)
        self.ctx, self.new, self.C, self.R, self.bs, self.dt, self.g = list(ctx), list(new), C, R, bs, dt, g
        need = [-(-(c + n) // bs) for c, n in zip(ctx, new)]
        self.num, W = sum(need) + 3, C + R
        order = torch.randperm(self.num, generator=g).to(torch.int32)
        self.table = torch.full((len(ctx), max(max(need), 1) + 1), -7, dtype=torch.int32)
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = order[at: at + k]
            at += k
        self.layout = layout
        self.pool = torch.full((self.num, bs, W), math.nan, dtype=dt)
        self.len = torch.tensor(ctx, dtype=torch.int32)
        self.cu = torch.tensor([0] + torch.tensor(list(new)).cumsum(0).tolist(), dtype=torch.int32)

    def slot(self, b, t):
        return int(self.table[b, t // self.bs]), t % self.bs

    def fill(self, spread=1.0):
        for b, (c, n) in enumerate(zip(self.ctx, self.new)):
            for j in range(-(-(c + n) // self.bs)):
                rows = min(self.bs, c + n - j * self.bs)
                x = torch.randn(rows, self.C + self.R, generator=self.g) * spread
                self.pool[int(self.table[b, j]), :rows] = x.to(self.dt)
        return self

    def entries(self, b):
        """[ctx + new, C + R] in 64 bits."""
        n = self.ctx[b] + self.new[b]
        if n == 0:
            return torch.zeros(0, self.C + self.R, dtype=torch.float64)
        ids = self.table[b, : -(-n // self.bs)].long()
        return self.pool[ids].flatten(0, 1)[:n].double()

    def to(self, dev):
        """The pool (by layout: dense, slots padded, or slots outside blocks), the table and the lengths."""
        W = self.C + self.R
        if self.layout == "padded":
            p = torch.full((self.num, self.bs + 1, W + 24), math.nan, dtype=self.dt, device=dev)[:, : self.bs, :W]
        elif self.layout == "slots":
            p = torch.full((self.bs, self.num, W), math.nan, dtype=self.dt, device=dev).transpose(0, 1)
        else:
            p = torch.empty(self.num, self.bs, W, dtype=self.dt, device=dev)
        p.copy_(self.pool)
        return p, self.table.to(dev), self.len.to(dev)


def attention(c: Cache, q, scale, mask=None):
    """The results, and what they may be off by, both [T, heads, C] in 64 bits.

    With half steps u of the type: the weights enter the second product rounded, relative by u, and their rounded sum divides:
    at most u / (1 - u) times sum p |v - o|. Scores are sums of W products in fp32, at most (W + 4) 2^-23 times sum |q e|
    scale off, which a weight takes as its relative error (and the exponential 2^-22). Sums over L slots in fp32 steps of 16:
    (L / 16 + 32) 2^-23 times sum p |v|. fp16 weights below 2^-14 of the reference, which no largest weight is below, are off
    by 2^-25 at most. The result is rounded once: u |o|, in fp16's subnormals 2^-25."""
    u = half_step(c.dt)
    out, tol, start = [], [], 0
    for b, (ctx, n) in enumerate(zip(c.ctx, c.new)):
        e = c.entries(b)
        v = e[:, : c.C]
        for i in range(n):
            see = torch.arange(ctx + n) < ctx
            step = mask[b, i, :n].bool() if mask is not None else torch.arange(n) <= i
            see[ctx:] = step
            for h in range(q.shape[1]):
                x = q[start + i, h].double()
                ev, vv = e[see], v[see]
                if ev.shape[0] == 0:
                    out.append(torch.zeros(c.C, dtype=torch.float64))
                    tol.append(torch.zeros(c.C, dtype=torch.float64))
                    continue
                p = torch.softmax(ev @ x * scale, 0)
                o = p @ vv
                apart, big = p @ (vv - o).abs(), p @ vv.abs()
                s = (ev.abs() @ x.abs()).max() * abs(scale) * (e.shape[1] + 4) * 2.0 ** -23 + 2.0 ** -22
                t = (u / (1 - u) + 2 * s) * apart + (ev.shape[0] / 16 + 32) * 2.0 ** -23 * big
                if c.dt == torch.float16:
                    t = t + 2.0 ** -25 * (1 + (vv - o).abs().sum(0))
                out.append(o)
                tol.append(t + u * (o.abs() + t))
        start += n
    shape = (start, q.shape[1], c.C)
    return (torch.stack(out).view(shape), torch.stack(tol).view(shape)) if out else (torch.zeros(shape), torch.zeros(shape))


def rotate(x, pos, freq, interleaved):
    x = x.double().clone()
    R = 2 * len(freq)
    for i, f in enumerate(freq):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        c, s = math.cos(pos * f), math.sin(pos * f)
        u, w = x[..., a].clone(), x[..., b].clone()
        x[..., a], x[..., b] = u * c - w * s, w * c + u * s
    return x


def normalise(x, w, eps):
    x = x.double()
    return x if w is None else x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()


def pages(table, length, refs, bs, keep=None, source=None, need=None):
    """The pages' update, step by step: rows, lengths, reference counts, statuses and the blocks copied."""
    B, M = table.shape
    old, refs = table.tolist(), refs.tolist()
    nb = len(refs)
    inside = lambda i: 0 <= i < nb  # noqa: E731
    rows, asks, bad = [], [], [False] * B
    for b in range(B):
        s = int(source[b]) if source is not None else b
        n = int(need[b]) if need is not None else 0
        sound = 0 <= s < B and n >= 0
        k = (int(keep[b]) if keep is not None else int(length[s])) if sound else 0
        sound = sound and 0 <= k <= int(length[s])
        bad[b] = not sound
        k, n = (k, n) if sound else (0, 0)
        kept = -(-k // bs)
        row = (old[s][:kept] if sound else []) + [-1] * (M - kept)
        bad[b] |= any(not inside(i) for i in row[:kept])
        rows.append(row)
        asks.append((k, kept, n))
    for b in range(B):
        for i in old[b]:
            if inside(i):
                refs[i] -= 1
        for i in rows[b]:
            if inside(i):
                refs[i] += 1
    at_start, free = list(refs), [i for i in range(nb) if refs[i] == 0]
    writers = {}
    for b, (k, kept, n) in enumerate(asks):
        if n and k % bs and -(-(k + n) // bs) <= M and inside(rows[b][kept - 1]):
            writers.setdefault(rows[b][kept - 1], []).append(b)
    copies, taken = [], 0
    for b, (k, kept, n) in enumerate(asks):
        if n == 0:
            continue
        blocks = -(-(k + n) // bs)
        if blocks > M:
            bad[b] = True
            continue
        last = rows[b][kept - 1] if kept else -1
        copy = b in writers.get(last, []) and at_start[last] >= 2 and \
            not (len(writers[last]) >= at_start[last] and writers[last][-1] == b)
        count = blocks - kept + copy
        taken += count
        if taken > len(free):
            bad[b] = True
            continue
        ids = free[taken - count: taken]
        rows[b][kept - copy: blocks] = ids
        for i in ids:
            refs[i] = 1
        if copy:
            refs[last] -= 1
            copies.append((last, ids[0]))
    return rows, [a[0] for a in asks], refs, [64 if x else 0 for x in bad], copies
