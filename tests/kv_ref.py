"""The cache operators of include/kv.h in 64-bit numpy, one sequence, head and row at a time, and the
inputs their tests share. Test infrastructure: shares no code with the CUDA path."""
from __future__ import annotations

import math

import numpy as np
import torch

from tests.gpu_util import canaries_intact, guarded

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
UNIT = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}  # largest relative rounding error


def host(t) -> np.ndarray:
    return t.detach().double().cpu().numpy() if t.is_floating_point() else t.detach().cpu().numpy()


def random_masks(r, B, T):
    """Mask words of random trees [B, T] (uint64)."""
    mask = np.zeros((B, T), np.uint64)
    for b in range(B):
        for i in range(T):
            parent = int(r.integers(-1, i)) if i else -1
            mask[b, i] = (mask[b, parent] if parent >= 0 else np.uint64(0)) | np.uint64(1) << np.uint64(i)
    return mask


def entries(pool, table, slot, h, n):
    """Rows 0..n-1 of a sequence from a pool [pages, Hkv, page_size, ...]."""
    ps = pool.shape[2]
    return np.stack([pool[table[slot, e // ps], h, e % ps] for e in range(n)]) if n else \
        np.zeros((0,) + pool.shape[3:], pool.dtype)


def attention(k, v, table, lengths, slots, q, kn, vn, mask, nodes, scale):
    """out, lse, and per output a bound's ingredients: sum p |v| and the largest sum |q k| scale of the row."""
    B, T, Hq, d = q.shape
    Hkv = kn.shape[2]
    G = Hq // Hkv
    out, lse = np.zeros((B, T, Hq, d)), np.full((B, T, Hq), -np.inf)
    mag, smag = np.zeros((B, T, Hq, d)), np.zeros((B, T, Hq))
    for b in range(B):
        slot = slots[b]
        if slot < 0:
            continue
        for h in range(Hkv):
            kc, vc = entries(k, table, slot, h, lengths[slot]), entries(v, table, slot, h, lengths[slot])
            for i in range(nodes[b]):
                seen = [j for j in range(nodes[b]) if int(mask[b, i]) >> j & 1]
                keys = np.concatenate([kc, kn[b, seen, h]]) if seen else kc
                vals = np.concatenate([vc, vn[b, seen, h]]) if seen else vc
                if len(keys) == 0:
                    continue
                for x in range(h * G, (h + 1) * G):
                    s = keys @ q[b, i, x] * scale
                    m = s.max()
                    e = np.exp(s - m)
                    lse[b, i, x] = m + math.log(e.sum())
                    p = e / e.sum()
                    out[b, i, x], mag[b, i, x] = p @ vals, p @ np.abs(vals)
                    smag[b, i, x] = (np.abs(keys) @ np.abs(q[b, i, x])).max() * abs(scale)
    return out, lse, mag, smag


def out_bound(mag, smag, d, dtype):
    """Each score is off by at most (d + 4) 2^-24 sum |q k| scale, which moves every weight by that share
    and their sum too; a 16-bit weight and the output are rounded once each; exponentials and divisions
    add a few 2^-22. Twice the rounding units plus 2^-19 covers them."""
    ds = (d + 4) * 2.0 ** -24 * smag[..., None] * 2
    return mag * (2 * UNIT[dtype] + 2 * ds + 2.0 ** -19) + (2.0 ** -24 if dtype == "f16" else 1e-30)


def lse_bound(lse, smag, d):
    return (d + 4) * 2.0 ** -24 * smag * 2 + 2.0 ** -20 * (1 + np.abs(np.where(np.isfinite(lse), lse, 0)))


def commit(c, table, lengths, counts, slots, kn, vn, path, npath):
    """Updates the dict c of pools (k, v, weights, stamps), lengths and counts in place."""
    ps = c["k"].shape[2]
    for b, slot in enumerate(slots):
        if slot < 0:
            continue
        for j in range(npath[b]):
            e = lengths[slot] + j
            pg, at = table[slot, e // ps], e % ps
            c["k"][pg, :, at], c["v"][pg, :, at] = kn[b, path[b, j]], vn[b, path[b, j]]
            c["weights"][pg, :, at], c["stamps"][pg, :, at] = 0, counts[slot] + j
        lengths[slot] += npath[b]
        counts[slot] += npath[b]


def accumulate(k, w, table, lengths, slots, q, lse, path, npath, scale, decay):
    """New weights (64 bits) and the bound on each."""
    w, tol = w.copy(), np.zeros(w.shape)
    B, T, Hq, d = q.shape
    Hkv, ps = k.shape[1], k.shape[2]
    G = Hq // Hkv
    for b, slot in enumerate(slots):
        if slot < 0 or npath[b] == 0:
            continue
        n, L = npath[b], lengths[slot]
        for h in range(Hkv):
            kc = entries(k, table, slot, h, L)
            add, off = np.zeros(L), np.zeros(L)
            for j in range(n):
                for x in range(h * G, (h + 1) * G):
                    z = lse[b, path[b, j], x]
                    if z == -np.inf:
                        continue
                    s = kc @ q[b, path[b, j], x] * scale
                    ds = (d + 4) * 2.0 ** -24 * (np.abs(kc) @ np.abs(q[b, path[b, j], x])) * abs(scale)
                    t = np.where(np.arange(L) <= L - n + j, np.exp(s - z), 0.0)
                    add += t
                    off += t * (2 * ds + 2.0 ** -21 * (2 + np.abs(s - z)))
            for e in range(L):
                i = (table[slot, e // ps], h, e % ps)
                w[i] = w[i] * decay + add[e]
                tol[i] = off[e] + 2.0 ** -22 * abs(w[i]) + 1e-37 + n * G * 2.0 ** -24 * add[e]
    return w, tol


def evict(c, table, lengths, counts, slots, budget, recent):
    """Updates the dict c of pools and lengths in place."""
    ps, Hkv = c["k"].shape[2], c["k"].shape[1]
    for slot in slots:
        if slot < 0 or lengths[slot] <= budget:
            continue
        L = lengths[slot]
        for h in range(Hkv):
            at = [(table[slot, e // ps], h, e % ps) for e in range(L)]

            def rank(e):  # ascending: best first
                w, st = c["weights"][at[e]], c["stamps"][at[e]]
                if st >= counts[slot] - recent:
                    return (0, 0.0, e)
                if np.isnan(w):
                    return (1, 0.0, e)
                return (2, -float(w), e)

            kept = set(sorted(range(L), key=rank)[:budget])
            holes = [e for e in range(budget) if e not in kept]
            fill = [e for e in range(budget, L) if e in kept]
            for to, fr in zip(holes, fill):
                for name in ("k", "v", "weights", "stamps"):
                    c[name][at[to]] = c[name][at[fr]]
        lengths[slot] = budget


def layout(shape, dtype, kind, device="cuda"):
    """Two pools [pages, Hkv, page_size, d] filled with NaN, in a memory layout of `kind`."""
    pages, H, ps, d = shape
    full = lambda *s: torch.full(s, float("nan"), dtype=TORCH[dtype], device=device)
    if kind == "heads":  # [page][head][place][d]
        return full(pages, H, ps, d), full(pages, H, ps, d)
    if kind == "places":  # [page][place][head][d]
        return full(pages, ps, H, d).transpose(1, 2), full(pages, ps, H, d).transpose(1, 2)
    if kind == "joint":  # keys and values of a place side by side
        x = full(pages, ps, H, 2, d)
        return x[..., 0, :].transpose(1, 2), x[..., 1, :].transpose(1, 2)
    assert kind == "odd"  # rows of d + 1 elements, off the 16-byte grid
    x, y = full(pages, H, ps, d + 1), full(pages, H, ps, d + 1)
    return x[..., 1:], y[..., 1:]


class Case:
    """A cache with sequences of the given lengths and, for each, T drafted nodes. Entries past a length,
    pages that nobody holds and nodes past a sequence's count are NaN."""

    def __init__(self, seed, dtype, lens, T, Hq, Hkv, d, page, nodes=None, kind="heads", room=0, pad=(), spread=1.0,
                 extra_slots=2):
        from hybrid_ssm_gated_gb300 import kv

        r = self.r = np.random.default_rng(seed)
        B = self.B = len(lens)
        self.T, self.Hq, self.Hkv, self.d, self.page, self.dtype = T, Hq, Hkv, d, page, dtype
        need = [-(-(n + room) // page) for n in lens]
        num_slots, num_pages, max_pages = B + extra_slots, sum(need) + 2, max(need + [1]) + 1
        self.slots = r.permutation(num_slots)[:B].astype(np.int32)
        order = r.permutation(num_pages)
        self.table = np.full((num_slots, max_pages), -7, np.int32)
        self.lengths = np.zeros(num_slots, np.int32)
        at = 0
        for b in range(B):
            self.table[self.slots[b], :need[b]] = order[at:at + need[b]]
            at += need[b]
            self.lengths[self.slots[b]] = lens[b]
        self.counts = self.lengths + 11
        for b in pad:
            self.slots[b] = -1
        self.k, self.v = layout((num_pages, Hkv, page, d), dtype, kind)
        for b in range(B):
            for e in range(lens[b]):
                if self.slots[b] >= 0:
                    pg = int(self.table[self.slots[b], e // page])
                    self.k[pg, :, e % page] = torch.from_numpy(r.normal(size=(Hkv, d)) * spread).to(self.k.dtype).cuda()
                    self.v[pg, :, e % page] = torch.from_numpy(r.normal(size=(Hkv, d))).to(self.k.dtype).cuda()
        self.nodes = np.array([T] * B if nodes is None else nodes, np.int32)
        rows = lambda H, s: torch.from_numpy(r.normal(size=(B, T, H, d)) * s).to(TORCH[dtype]).cuda()
        self.q, self.kn, self.vn = rows(Hq, spread), rows(Hkv, spread), rows(Hkv, 1.0)
        for b in range(B):
            for x in (self.q, self.kn, self.vn):
                x[b, max(int(self.nodes[b]), 0):] = float("nan")
        self.mask = random_masks(r, B, T)
        shape = (num_pages, Hkv, page)
        self.weights = torch.from_numpy(r.exponential(size=shape)).float().cuda()
        self.stamps = torch.from_numpy(r.integers(0, 9, size=shape)).int().cuda()
        self.kv = kv
        self.scale = 1.0 / math.sqrt(d)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.sync()

    def sync(self):
        """Device copies of the host's bookkeeping, and the cache handle."""
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
        self.d_slots, self.d_nodes = dev(self.slots), dev(self.nodes)
        self.d_mask = dev(self.mask.view(np.int64))
        self.d_lengths, self.d_counts = dev(self.lengths), dev(self.counts)
        self.cache = self.kv.KVCache(self.k, self.v, dev(self.table), self.d_lengths, self.d_counts, self.weights,
                                     self.stamps)

    def attend(self, stream=None, with_nodes=True, with_lse=True):
        guards = []  # poisoned bytes around everything the call writes
        out = guarded(self.q.shape, self.q.dtype, guards).fill_(7.0)
        lse = guarded(self.q.shape[:3], torch.float32, guards).fill_(7.0) if with_lse else None
        ws = guarded((self.kv.kv_tree_workspace(self.cache, self.q).numel(),), torch.uint8, guards).fill_(0xFF)
        torch.cuda.synchronize()
        self.kv.kv_tree_attention(self.cache, self.d_slots, self.q, self.kn, self.vn, self.d_mask, out, self.err, ws,
                                  num_nodes=self.d_nodes if with_nodes else None, lse=lse, scale=self.scale,
                                  stream=stream)
        torch.cuda.synchronize()
        assert canaries_intact(guards)
        return out, lse

    def reference(self):
        return attention(host(self.k), host(self.v), self.table, self.lengths, self.slots, host(self.q), host(self.kn),
                         host(self.vn), self.mask, self.nodes, self.scale)

    def check_attention(self, expect_err=0):
        out, lse = self.attend()
        ref, rl, mag, smag = self.reference()
        assert int(self.err.item()) == expect_err
        o, z = host(out), host(lse)
        bad = np.abs(o - ref) > out_bound(mag, smag, self.d, self.dtype)
        assert not bad.any() and not np.isnan(o).any(), f"{bad.sum()} outputs off, by {np.nanmax(np.abs(o - ref)):.3e}"
        assert np.array_equal(np.isneginf(z), np.isneginf(rl))
        fin = np.isfinite(rl)
        off = np.abs(z[fin] - rl[fin])
        assert (off <= lse_bound(rl, smag, self.d)[fin]).all(), f"lse off by {off.max():.3e}"
        return out, lse

    def pools(self):
        """Host copies of what a cache holds."""
        return {"k": host(self.k), "v": host(self.v), "weights": self.weights.cpu().numpy().copy(),
                "stamps": self.stamps.cpu().numpy().copy()}

    def assert_pools(self, want):
        for name, x in (("k", self.k), ("v", self.v)):
            assert np.array_equal(host(x), want[name], equal_nan=True), name
        assert np.array_equal(self.weights.cpu().numpy(), want["weights"], equal_nan=True)
        assert np.array_equal(self.stamps.cpu().numpy(), want["stamps"])
