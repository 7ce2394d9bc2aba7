"""Tree verification steps of several samples of one prompt, on a paged latent cache.

The target keeps one latent vector a token, of which every head asks in its own way. It is a small associative memory: a
token's latent vector is the name of the token before it next to its own value, so that asking with a token's name answers
with the token that follows it, which the prompt alone knows. One prompt is prefilled; then the other sequences are forked
from it, its blocks are shared, and the partly filled last one is copied before it is written. Every step

  1. gives back the blocks of rejected tokens and takes those of the next tree    (spec_pages_update),
  2. merges two drafters' trees on the device                                      (spec_merge_trees),
  3. normalises and appends the nodes' latent vectors, rotates keys and queries    (spec_latent_append), a layer at a time,
  4. attends over cache and tree under the merged mask                             (spec_latent_attention),
  5. takes the longest path that the target agrees with                            (spec_verify_tree_greedy),
  6. keeps that path's entries in all layers                                       (spec_latent_compact).

    python examples/latent_step.py [--steps 30]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import speculative_decoding_verification_29_gb300 as sv  # noqa: E402
from tree_step import NODES, PARENT, shape  # noqa: E402

LAYERS, HEADS, LATENT, ROT, BLOCK = 2, 8, 256, 32, 16
INV_FREQ = [10000.0 ** (-i / 16) for i in range(16)]
TOKENS = 41
HALF = LATENT // 2  # names in the first half of the latent vector, values in the second


class Target:
    def __init__(self, B, longest, seed, dev):
        g = torch.Generator().manual_seed(seed)
        self.B, self.dev, self.g = B, dev, g
        sign = lambda *s: (torch.randint(0, 2, s, generator=g).float() * 2 - 1).to(dev)  # noqa: E731
        self.names, self.values = sign(TOKENS, LAYERS, HALF), sign(TOKENS, LAYERS, HALF)
        order = torch.randperm(TOKENS, generator=g)  # one cycle over all tokens
        self.next = torch.empty(TOKENS, dtype=torch.long)
        self.next[order] = order.roll(-1)
        self.width = -(-longest // BLOCK)
        blocks = B * self.width
        self.pool = torch.zeros(LAYERS, blocks, BLOCK, LATENT + ROT, dtype=torch.bfloat16, device=dev)
        self.table = torch.full((B, self.width), -1, dtype=torch.int32, device=dev)
        self.refs = torch.zeros(blocks, dtype=torch.int32, device=dev)
        self.len = torch.zeros(B, dtype=torch.int32, device=dev)

    def pages(self, need, source=None):
        """Rows for `need` more tokens each, of the sequences themselves or forked."""
        need = torch.tensor(need, dtype=torch.int32, device=self.dev)
        source = None if source is None else torch.tensor(source, dtype=torch.int32, device=self.dev)
        r = sv.spec_pages_update(self.table, self.len, self.refs, [self.pool], planes=True, source=source, need=need)
        assert not bool(r["row_status"].any())
        self.table, self.len = r["block_table"], r["cache_len"]

    def forward(self, asks, names, tokens, cu, max_tokens, strength, positions=None, mask=None):
        """One pass over packed tokens: the cache grows by (names -> tokens), the answers' logits return."""
        logits = 0
        for layer in range(LAYERS):
            x = torch.cat((self.names[names, layer], self.values[tokens, layer]), -1).bfloat16() * 3.0
            weight = torch.full((LATENT,), strength, device=self.dev)  # the norm takes the 3 out, the weight remains
            q = torch.zeros(len(asks), HEADS, LATENT + ROT, dtype=torch.bfloat16, device=self.dev)
            q[..., :HALF] = self.names[asks, layer][:, None]
            q[..., LATENT:] = 0.05
            rope = torch.full((len(asks), ROT), 0.05, dtype=torch.bfloat16, device=self.dev)
            tail = q[..., LATENT:]
            r = sv.spec_latent_append(x, rope, self.pool[layer], self.table, self.len, cu, inv_freq=INV_FREQ, positions=positions,
                                      norm_weight=weight, q_rope=tail, q_out=tail)
            o = sv.spec_latent_attention(q, self.pool[layer], self.table, self.len, cu, max_tokens=max_tokens, value_dim=LATENT,
                                         sm_scale=0.25, tree_mask=mask)
            assert not bool((r["row_status"] | o["row_status"]).any())
            logits = logits + o["out"][..., HALF:].float().mean(1) @ self.values[:, layer].T
        return logits

    def prompt(self):
        """The first sequence reads the prompt, every token and its successor once; the others become its forks."""
        a = torch.randperm(TOKENS, generator=self.g)
        self.pages([TOKENS] + [0] * (self.B - 1))
        cu = torch.tensor([0] + [TOKENS] * self.B, dtype=torch.int32, device=self.dev)
        self.forward(a.to(self.dev), a.to(self.dev), self.next[a].to(self.dev), cu, TOKENS, 1.0)
        self.len[0] += TOKENS


def draft(target, root, parent, p_right, rng):
    """A drafter's tokens: a node is its parent's successor with probability p_right, else any token."""
    tok = torch.zeros(target.B, len(parent), dtype=torch.long)
    tok[:, 0] = root
    for i, p in enumerate(parent[1:], 1):
        guess = torch.randint(0, TOKENS, (target.B,), generator=rng)
        tok[:, i] = torch.where(torch.rand(target.B, generator=rng) < p_right, target.next[tok[:, p]], guess)
    return tok


def run(steps=30, B=4, seed=0, device="cuda:0"):
    """The tokens that every sequence emitted, the right ones, the mean number a step emitted, and the target."""
    dev = torch.device(device)
    n = 2 * NODES + 1
    target = Target(B, TOKENS + steps * 8 + n, seed, dev)
    target.prompt()
    rng = torch.Generator().manual_seed(seed + 1)
    root = torch.randint(0, TOKENS, (B,), generator=rng)
    before = torch.empty(TOKENS, dtype=torch.long)
    before[target.next] = torch.arange(TOKENS)
    prev = before[root]  # the token before the root, which the root's entry names
    shapes = [shape(p) for p in PARENT]
    merged = torch.tensor(PARENT[0] + [p + NODES if p > 0 else p for p in PARENT[1][1:]], device=dev)
    cu = torch.arange(B + 1, dtype=torch.int32, device=dev) * n
    emitted, right = [[] for _ in range(B)], [[] for _ in range(B)]
    source = [0] * B  # the first step forks the prompt
    for _ in range(steps):
        target.pages([n] * B, source)
        source = None
        trees = []
        for (mask, rows, depth), parent, p_right in zip(shapes, PARENT, (0.7, 0.5)):
            tok = draft(target, root, parent, p_right, rng).int()
            trees += [t.to(dev) for t in (tok, mask.expand(B, -1, -1), rows.expand(B, -1, -1), depth.expand(B, -1))]
        m = sv.spec_merge_trees(*trees)
        tok = m["tokens"].long()
        names = torch.where(merged[None] >= 0, tok[:, merged.clamp(min=0)], prev[:, None].to(dev))
        logits = target.forward(tok.flatten(), names.flatten(), tok.flatten(), cu, n, 1.1,
                                (target.len[:, None] + m["pos"]).flatten(), m["mask"]).view(B, n, TOKENS)
        r = sv.spec_verify_tree_greedy(logits, m["tokens"], m["retrieve"], m["n1"], tree_mask=m["mask"])
        c = sv.spec_latent_compact(target.pool, target.table, target.len, r["accept_len"], r["path_nodes"])
        assert not bool((r["row_status"] | c["row_status"]).any())
        target.len = c["new_len"]
        out = r["out_tokens"].cpu()
        for b in range(B):
            for x in out[b].tolist():
                if x >= 0:
                    right[b].append(int(target.next[int(root[b])]))
                    prev[b], root[b] = root[b], x
                    emitted[b].append(x)
    return emitted, right, sum(map(len, emitted)) / (B * steps), target


if __name__ == "__main__":
    args = argparse.ArgumentParser()
    args.add_argument("--steps", type=int, default=30)
    emitted, right, mean, _ = run(args.parse_args().steps)
    print(f"{sum(map(len, emitted))} tokens emitted, {mean:.2f} a step and sequence, "
          f"{'all right' if emitted == right else 'NOT all right'}")
    sys.exit(emitted != right)
