"""Speculative decoding of a small hybrid model with draft trees: a Gated DeltaNet layer and an attention
layer, random weights, greedy choice.

Each round drafts a tree of tokens behind every sequence's last token and verifies it in one pass:
  - the recurrent layer runs the tree level by level with gdn_spec_step, a node's state going from its
    parent's slot to its own, so no state is taken back when a draft is rejected;
  - the attention layer runs it at once with kv_tree_attention over the paged cache and the tree's mask.
The accepted path then becomes the sequence: kv_commit appends its keys and values, the sequence takes
over the recurrent state slot of its last node, kv_accumulate adds the attention weight that the accepted
tokens gave to the cache's entries, and kv_evict brings caches past their budget back to it.

Without a budget the result is, token for token, that of decoding one token at a time (the same calls with
a tree of one node), which main() checks:  python examples/hybrid_tree_verify.py
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from hybrid_ssm_gated_gb300 import gdn, kv  # noqa: E402

VOCAB, WIDTH = 24, 256
HK, HV, DK, DV = 2, 4, 64, 64  # recurrent layer
HQ, HKV, D, PAGE = 8, 2, 64, 16  # attention layer


class Model:
    """Random weights of the two layers, and their projections."""

    def __init__(self, seed: int):
        g = torch.Generator().manual_seed(seed)
        w = lambda *s: (torch.randn(*s, generator=g) / math.sqrt(s[0])).cuda()
        self.embedding = torch.randn(VOCAB, WIDTH, generator=g).cuda()
        self.in_gdn, self.out_gdn = w(WIDTH, (2 * HK * DK) + HV * DV + 2 * HV), w(HV * DV, WIDTH)
        self.in_attn, self.out_attn = w(WIDTH, (HQ + 2 * HKV) * D), w(HQ * D, WIDTH)
        self.head = w(WIDTH, VOCAB)
        self.A_log, self.dt_bias = torch.rand(HV, generator=g).cuda(), torch.zeros(HV, device="cuda")

    @staticmethod
    def norm(x):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)

    @staticmethod
    def rotate(x, position):
        """Rotary embedding of x [B, N, H, D] at positions [B, N]."""
        f = 10000.0 ** (-torch.arange(0, D, 2, device=x.device) / D)
        a = position[..., None, None].float() * f
        x1, x2 = x[..., 0::2], x[..., 1::2]
        return torch.stack((x1 * a.cos() - x2 * a.sin(), x1 * a.sin() + x2 * a.cos()), -1).flatten(-2)


class Decoder:
    """Sequences in decoding: recurrent state slots, a paged cache, and each sequence's last token."""

    def __init__(self, model: Model, tokens, nodes: int, capacity: int, budget: int = 0, recent: int = 0):
        self.m, self.B, self.N, self.budget, self.recent = model, len(tokens), nodes, budget, recent
        per = -(-capacity // PAGE)
        self.last = torch.tensor(tokens, device="cuda")
        # a state slot for each sequence and one for each node of a tree: [B, 1 + N]
        self.state = torch.zeros(self.B * (1 + nodes), HV, DV, DK, device="cuda")
        self.state_slots = torch.arange(self.B * (1 + nodes), dtype=torch.int32, device="cuda").view(self.B, 1 + nodes)
        self.cache = kv.KVCache.allocate(self.B * per, HKV, PAGE, D, self.B, per, torch.float32)
        self.cache.page_table.copy_(torch.arange(self.B * per, dtype=torch.int32).view(self.B, per))
        self.slots = torch.arange(self.B, dtype=torch.int32, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.work = None
        self.evict_work = kv.kv_evict_workspace(self.cache, self.B, budget) if budget else None

    def recurrent(self, x, depth, parent):
        """The recurrent layer over the tree's nodes [B, N, WIDTH], level by level."""
        y = self.m.norm(x) @ self.m.in_gdn
        q, k, v, a, b = y.split([HK * DK, HK * DK, HV * DV, HV, HV], -1)
        out = torch.empty(x.shape[0], x.shape[1], HV, DV, device="cuda")
        for level in range(int(depth.max()) + 1):
            at = [i for i in range(x.shape[1]) if depth[i] == level]
            take = lambda t, *s: t[:, at].reshape(-1, 1, *s).contiguous()
            src = torch.stack([self.state_slots[:, 0 if parent[i] < 0 else 1 + parent[i]] for i in at], 1)
            dst = torch.stack([self.state_slots[:, 1 + i] for i in at], 1)
            o = torch.empty(self.B * len(at), 1, HV, DV, device="cuda")
            gdn.gdn_spec_step(self.state, src.reshape(-1).contiguous(), dst.reshape(-1, 1).contiguous(), take(q, HK, DK),
                              take(k, HK, DK), take(v, HV, DV), take(a, HV), take(b, HV), self.m.A_log, self.m.dt_bias, o,
                              self.err)
            out[:, at] = o.view(self.B, len(at), HV, DV)
        return x + out.flatten(2) @ self.m.out_gdn

    def verify(self, tokens, parent):
        """One pass over a tree of tokens [B, N] (node 0: the last token): the greedy choice after each
        node [B, N], and what the commit takes."""
        parent = list(parent)
        depth = torch.zeros(len(parent), dtype=torch.long)
        for i, p in enumerate(parent):
            depth[i] = 0 if p < 0 else depth[p] + 1
        x = self.recurrent(self.m.embedding[tokens], depth, parent)
        qkv = (self.m.norm(x) @ self.m.in_attn).unflatten(-1, (HQ + 2 * HKV, D))
        position = self.cache.counts[self.slots.long()][:, None] + depth.cuda()
        qkv[:, :, :HQ + HKV] = self.m.rotate(qkv[:, :, :HQ + HKV], position)
        q, k, v = qkv.split([HQ, HKV, HKV], 2)  # parts of one projection: the cache's calls take strides
        mask = kv.tree_masks([parent] * self.B).cuda()
        out, lse = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:3], device="cuda")
        if self.work is None:
            self.work = kv.kv_tree_workspace(self.cache, q)
        kv.kv_tree_attention(self.cache, self.slots, q, k, v, mask, out, self.err, self.work, lse=lse)
        x = x + out.flatten(2) @ self.m.out_attn
        return (self.m.norm(x) @ self.m.head).argmax(-1), (q, k, v, lse)

    def accept(self, path, n_path, made):
        """The accepted paths [B, P] (n_path [B] nodes of them) become the sequences."""
        q, k, v, lse = made
        path, n_path = path.int().cuda(), n_path.int().cuda()
        kv.kv_commit(self.cache, self.slots, k, v, path, n_path, self.err)
        kv.kv_accumulate(self.cache, self.slots, q, lse, path, n_path, self.err)
        if self.budget:
            kv.kv_evict(self.cache, self.slots, self.budget, self.recent, self.err, self.evict_work)
        # the state after the last accepted node: the sequence and that node change slots
        leaf = path.gather(1, (n_path.long() - 1)[:, None]) + 1
        mine, its = self.state_slots[:, :1].clone(), self.state_slots.gather(1, leaf.long())
        self.state_slots.scatter_(1, leaf.long(), mine)
        self.state_slots[:, :1] = its

    def decode(self, steps: int):
        """Greedy tokens [B, steps], one at a time: trees of one node."""
        made = []
        one = torch.zeros(self.B, 1), torch.ones(self.B)
        for _ in range(steps):
            choice, rows = self.verify(self.last[:, None], [-1])
            self.accept(*one, rows)
            self.last = choice[:, 0]
            made.append(self.last)
        return torch.stack(made, 1)

    def speculate(self, steps: int, guess):
        """Greedy tokens of each sequence (at least `steps`) from verified trees; guess(round) gives a tree's
        parents and the tokens drafted for its nodes 1 .. N - 1 [B, N - 1]."""
        made, rounds = [[] for _ in range(self.B)], 0
        while min(map(len, made)) < steps:
            parent, drafts = guess(rounds)
            tokens = torch.cat([self.last[:, None], drafts.cuda()], 1)
            choice, rows = self.verify(tokens, parent)
            path, n_path = torch.zeros(self.B, len(parent)), torch.ones(self.B)
            said, wanted = tokens.tolist(), choice.tolist()
            for b in range(self.B):
                node = 0
                while True:
                    made[b].append(wanted[b][node])
                    hit = [i for i, p in enumerate(parent) if p == node and said[b][i] == wanted[b][node]]
                    if not hit:
                        break
                    node = hit[0]
                    path[b, int(n_path[b])] = node
                    n_path[b] += 1
            self.accept(path, n_path, rows)
            self.last = torch.tensor([m[-1] for m in made], device="cuda")
            rounds += 1
        return [m[:steps] for m in made], rounds


def guesses(truth, seed: int, parent=(-1, 0, 0, 1, 1, 2, 3)):
    """Drafts for a run whose continuation is known: each node holds the right token two times in three."""
    g = torch.Generator().manual_seed(seed)

    def guess(made):
        depth = [0] * len(parent)
        for i, p in enumerate(parent):
            depth[i] = 0 if p < 0 else depth[p] + 1
        rows = []
        for b, done in enumerate(made()):
            right = lambda i: truth[b][min(done + depth[i] - 1, len(truth[b]) - 1)]
            rows.append([right(i) if torch.rand(1, generator=g) < 0.67 else int(torch.randint(VOCAB, (1,), generator=g))
                         for i in range(1, len(parent))])
        return list(parent), torch.tensor(rows)

    return guess


def run(batch: int = 3, steps: int = 60, budget: int = 0, recent: int = 0, seed: int = 1):
    """Tokens decoded one at a time, tokens from verified trees, rounds of the latter, its decoder."""
    model = Model(seed)
    first = [i % VOCAB for i in range(batch)]
    plain = Decoder(model, first, 1, steps + 40).decode(steps + 16).tolist()
    tree = Decoder(model, first, 7, steps + 40, budget, recent)
    draft = guesses(plain, seed)
    lengths = lambda: tree.cache.counts.tolist()
    said, rounds = tree.speculate(steps, lambda _: draft(lengths))
    return [p[:steps] for p in plain], said, rounds, tree


def main():
    plain, said, rounds, tree = run()
    assert int(tree.err.item()) == 0, f"device error word {int(tree.err.item())}"
    assert plain == said, "the verified trees gave other tokens than decoding one at a time"
    print(f"{len(said[0])} tokens a sequence in {rounds} rounds, the same as one at a time")
    _, said, rounds, tree = run(budget=32, recent=8)
    assert int(tree.err.item()) == 0, f"device error word {int(tree.err.item())}"
    print(f"with caches of 32 entries: lengths {tree.cache.lengths.tolist()} after {tree.cache.counts.tolist()} tokens")


if __name__ == "__main__":
    main()
