"""The cached attention's 64-bit form with tolerances of the kernel that takes the rows, which rows 2^14 times larger beside a
row hardly widen."""

from __future__ import annotations

import math

import torch

import kv8_plain as plain


def attention(c: plain.Cache, q, scale, max_tokens, tree=None):
    """(out, tolerance) [T, Hq, D] in 64 bits for q's type.

    A result o = sum_t p_t v_t, A = sum_t p_t |v_t|, is off by
    - half a step of the output's type on o;
    - the weights' rounding relative to A. Up to 64 rows (max_tokens times the query heads of a KV head): two e4m3 terms for
      bf16 (2^-4 of 2^-4), three for fp16 (2^-11). Above: fp16, 2^-11;
    - the weights' floor. Up to 64 rows, in each tile of 128: half of e4m3's least step 2^-9 where the tile's largest weight
      is above 2^7, so 2^-17 of that weight for each slot. Above: half of fp16's least step 2^-24 where the row's largest
      weight is at least 2^-1, so 2^-24 of that weight for each slot;
    - the scores' error ds, which moves the weights by 2 ds. Queries are exact down to a floor, half of the least step over
      the largest element. Up to 64 rows: of the sequence's rows of the KV head, e5m2 2^-17 over 28672 (< 2^-31). Above: of
      the row, fp16 2^-25 over 2^13 (2^-38). The products' sums take 2^-20 of sum |q k|;
    - the exponent's and the sums' rounding in fp32: exponents are below 2^6 + the scores' bits, 2^-17 of A with the sums."""
    bf = q.dtype == torch.bfloat16
    T, Hq, D = q.shape
    g = Hq // c.H
    wide = max_tokens * g > 64
    half = 2.0 ** -8 if bf else 2.0 ** -11
    wrel, wfloor = (2.0 ** -11, 2.0 ** -24) if wide else (2.0 ** -8 if bf else 2.0 ** -11, 2.0 ** -17)
    out, tol = torch.full((T, Hq, D), math.nan, dtype=torch.float64), torch.zeros(T, Hq, D, dtype=torch.float64)
    for b, (ctx, n) in enumerate(zip(c.ctx, c.new)):
        if not n:
            continue
        t0, L = int(c.cu[b]), ctx + n
        k, _, _ = c.rows(c.k, c.ks, b, L)
        v, vraw, vexp = c.rows(c.v, c.vs, b, L)
        seen = torch.ones(n, L, dtype=torch.bool)
        seen[:, ctx:] = tree[b, :n, :n].bool() if tree is not None else torch.ones(n, n).tril().bool()
        pad = -L % plain.TILE
        for a in range(Hq):
            h = a // g
            x = q[t0: t0 + n, a].double()  # [n, D]
            w = ((x @ k[h].T) * scale).masked_fill(~seen, -math.inf)
            p = torch.softmax(w, -1).nan_to_num(0.0)  # rows that see nothing
            o, A = p @ v[h], p @ v[h].abs()
            own, largest = x.abs().amax(-1, keepdim=True), q[t0: t0 + n, h * g: (h + 1) * g].double().abs().max()
            qfloor = own * 2.0 ** -38 if wide else largest * 2.0 ** -31
            qk = (k[h].abs().sum(-1) * qfloor + (x.abs() @ k[h].abs().T) * 2.0 ** -20)
            ds = abs(scale) * (qk * seen).amax(-1, keepdim=True)
            wt = p * torch.pow(2.0, vexp[h])
            codes = vraw[h].abs()
            if wide:
                floor = wt.amax(-1, keepdim=True) * (seen.double() @ codes)
            else:
                tiles = torch.nn.functional.pad(wt, (0, pad)).view(n, -1, plain.TILE).amax(-1)
                of = torch.nn.functional.pad(seen.double(), (0, pad)).view(n, -1, plain.TILE)
                floor = torch.einsum("nt,nts,tsd->nd", tiles, of, torch.nn.functional.pad(codes, (0, 0, 0, pad)).view(
                    -1, plain.TILE, D))
            out[t0: t0 + n, a] = o
            tol[t0: t0 + n, a] = o.abs() * half * 1.01 + A * (wrel + 2 * ds + 2.0 ** -17) + floor * wfloor + 1e-30
            if not bf:
                tol[t0: t0 + n, a] += 2.0 ** -25  # fp16's least step, halved
    return out, tol


def check(c, q, got, status, scale, max_tokens, tree=None):
    want, tol = attention(c, q, scale, max_tokens, tree)
    assert status == [0] * len(c.ctx)
    assert not torch.isnan(got).any()
    rel = (got - want).abs() / tol
    bad = rel > 1
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {float(rel.max()):.2f} tolerances"
