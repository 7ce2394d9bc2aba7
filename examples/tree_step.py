"""Tree verification steps on an 8-bit paged KV cache, as a serving loop runs them.

The target is a small associative memory, so that the right answer is known. A prompt token is a pair (a -> next(a)) of a
permutation: its key names a and its value names next(a), in every layer and KV head with other random codes. Decoding
token a asks with the query of a and has to answer next(a), so the model walks the permutation, which only its cache
knows. Two drafters propose a tree each, with right and wrong guesses. Every step

  1. merges the trees on the device                       (spec_merge_trees),
  2. rotates and appends the nodes' keys and values       (spec_kv8_append), a layer at a time,
  3. attends over cache and tree under the merged mask    (spec_kv8_attention),
  4. takes the longest path that the target agrees with   (spec_verify_tree_greedy),
  5. keeps that path's entries in all layers              (spec_kv8_compact).

A node's entry names its parent as key and itself as value, and is stronger than the prompt's: a mask or a compaction that
leaks a wrong guess would answer with it.

    python examples/tree_step.py [--steps 40]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_29_gb300 as sv  # noqa: E402

LAYERS, Q_HEADS, KV_HEADS, HEAD_DIM, BLOCK = 2, 8, 2, 128, 16
ROT, INV_FREQ = 32, [10000.0 ** (-i / 16) for i in range(16)]
TOKENS = 41
NODES = 6  # each drafter's nodes below the root
PARENT = [[-1, 0, 1, 2, 0, 4, 5], [-1, 0, 0, 1, 2, 3, 4]]  # the drafters' tree shapes


def shape(parent):
    """Ancestor mask, retrieve rows and depths of a tree."""
    n = len(parent)
    mask, depth = torch.zeros(n, n, dtype=torch.uint8), torch.zeros(n, dtype=torch.int32)
    for i, p in enumerate(parent):
        if p >= 0:
            mask[i], depth[i] = mask[p], depth[p] + 1
        mask[i, i] = 1
    leaves = [i for i in range(n) if i not in parent]
    rows = torch.full((len(leaves), int(depth.max()) + 1), -1, dtype=torch.int32)
    for r, leaf in enumerate(leaves):
        while leaf >= 0:
            rows[r, depth[leaf]] = leaf
            leaf = parent[leaf]
    return mask, rows, depth


class Target:
    def __init__(self, B, longest, seed, dev):
        g = torch.Generator().manual_seed(seed)
        self.B, self.dev, self.g = B, dev, g
        sign = lambda *s: torch.randint(0, 2, s, generator=g).float() * 2 - 1  # noqa: E731
        names = sign(TOKENS, LAYERS, KV_HEADS, HEAD_DIM)
        names[..., :ROT] *= 0.1  # the rotated part: positions stir the scores a little
        self.names, self.values = names.to(dev, torch.bfloat16), sign(TOKENS, LAYERS, KV_HEADS, HEAD_DIM).to(dev, torch.bfloat16)
        order = torch.stack([torch.randperm(TOKENS, generator=g) for _ in range(B)])  # one cycle per sequence
        self.next = torch.empty(B, TOKENS, dtype=torch.long)
        self.next.scatter_(1, order, order.roll(-1, 1))
        per = -(-longest // BLOCK)
        pool = (LAYERS, B * per, KV_HEADS, BLOCK, HEAD_DIM)
        self.k, self.v = (torch.zeros(pool, dtype=torch.uint8, device=dev) for _ in range(2))
        self.ks, self.vs = (torch.zeros(pool[:3], dtype=torch.uint8, device=dev) for _ in range(2))
        self.table = torch.randperm(B * per, generator=g).view(B, per).to(dev, torch.int32)
        self.len = torch.zeros(B, dtype=torch.int32, device=dev)

    def cache(self, layer):
        return self.k[layer], self.v[layer], self.ks[layer], self.vs[layer], self.table, self.len

    def forward(self, asks, keys, values, strength, max_tokens, positions=None, mask=None):
        """One pass over packed tokens [B * max_tokens]: the cache grows by (keys -> values), the answers' logits return."""
        cu = torch.arange(self.B + 1, dtype=torch.int32, device=self.dev) * max_tokens
        logits = 0
        for layer in range(LAYERS):
            q = self.names[asks, layer].repeat_interleave(Q_HEADS // KV_HEADS, 1)
            r = sv.spec_kv8_append(self.names[keys, layer] * strength, self.values[values, layer], *self.cache(layer), cu,
                                   inv_freq=INV_FREQ, positions=positions, q=q)
            o = sv.spec_kv8_attention(r["q_out"], *self.cache(layer), cu, max_tokens=max_tokens, sm_scale=0.25,
                                      tree_mask=mask)
            assert not bool((r["row_status"] | o["row_status"]).any())
            heads = self.values[:, layer].repeat_interleave(Q_HEADS // KV_HEADS, 1).flatten(1)
            logits = logits + o["out"].flatten(1).float() @ heads.float().T
        return logits.view(self.B, max_tokens, TOKENS)

    def prompt(self):
        a = torch.stack([torch.randperm(TOKENS, generator=self.g) for _ in range(self.B)])
        b = self.next.gather(1, a)
        a, b = a.flatten().to(self.dev), b.flatten().to(self.dev)
        self.forward(a, a, b, 1.0, TOKENS)
        self.len += TOKENS


def draft(target, root, parent, p_right, rng):
    """A drafter's tokens: a node is its parent's successor with probability p_right, else any token."""
    tok = torch.zeros(target.B, len(parent), dtype=torch.long)
    tok[:, 0] = root
    for i, p in enumerate(parent[1:], 1):
        right = target.next.gather(1, tok[:, p: p + 1])[:, 0]
        guess = torch.randint(0, TOKENS, (target.B,), generator=rng)
        tok[:, i] = torch.where(torch.rand(target.B, generator=rng) < p_right, right, guess)
    return tok


def run(steps=40, B=4, seed=0, device="cuda:0"):
    """The tokens that every sequence emitted, the right ones, and the mean number a step emitted."""
    dev = torch.device(device)
    n = 2 * NODES + 1
    target = Target(B, TOKENS + steps * 8 + n, seed, dev)
    target.prompt()
    rng = torch.Generator().manual_seed(seed + 1)
    root = torch.randint(0, TOKENS, (B,), generator=rng)
    came_from = torch.empty(B, TOKENS, dtype=torch.long).scatter_(1, target.next, torch.arange(TOKENS).expand(B, -1))
    prev = came_from.gather(1, root[:, None])[:, 0]  # the token before the root, which the root's entry names
    shapes = [shape(p) for p in PARENT]
    merged_parent = torch.tensor(PARENT[0] + [p + NODES if p > 0 else p for p in PARENT[1][1:]])
    emitted, right = [[] for _ in range(B)], [[] for _ in range(B)]
    for _ in range(steps):
        trees = []
        for (mask, rows, depth), parent, p_right in zip(shapes, PARENT, (0.7, 0.5)):
            tok = draft(target, root, parent, p_right, rng).int()
            trees += [t.to(dev) for t in (tok, mask.expand(B, -1, -1), rows.expand(B, -1, -1), depth.expand(B, -1))]
        m = sv.spec_merge_trees(*trees)
        tok = m["tokens"].long()
        parents = torch.where(merged_parent[None].to(dev) >= 0, tok[:, merged_parent.clamp(min=0).to(dev)],
                              prev[:, None].to(dev))
        logits = target.forward(tok.flatten(), parents.flatten(), tok.flatten(), 1.25, n,
                                (target.len[:, None] + m["pos"]).flatten(), m["mask"])
        r = sv.spec_verify_tree_greedy(logits, m["tokens"], m["retrieve"], m["n1"], tree_mask=m["mask"])
        c = sv.spec_kv8_compact(target.k, target.v, target.ks, target.vs, target.table, target.len, r["accept_len"],
                                r["path_nodes"])
        assert not bool((r["row_status"] | c["row_status"]).any())
        target.len = c["new_len"]
        out = r["out_tokens"].cpu()
        for b in range(B):
            for x in out[b].tolist():
                if x >= 0:
                    right[b].append(int(target.next[b, int(root[b])]))
                    prev[b], root[b] = root[b], x
                    emitted[b].append(x)
    return emitted, right, sum(map(len, emitted)) / (B * steps)


if __name__ == "__main__":
    args = argparse.ArgumentParser()
    args.add_argument("--steps", type=int, default=40)
    emitted, right, mean = run(args.parse_args().steps)
    print(f"{sum(map(len, emitted))} tokens emitted, {mean:.2f} a step and sequence, "
          f"{'all right' if emitted == right else 'NOT all right'}")
    sys.exit(emitted != right)
