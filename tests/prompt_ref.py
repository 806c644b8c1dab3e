"""The prompt and page operators of include/kv.h in 64-bit numpy, and the inputs their tests share. Test
infrastructure: shares no code with the CUDA path."""
from __future__ import annotations

import math

import numpy as np
import torch

from tests.gpu_util import canaries_intact, guarded
from tests.kv_ref import TORCH, UNIT, entries, host, layout, lse_bound, out_bound


def turned(x, weight, eps, offset, freq, axis, positions, interleaved):
    """Rows x [tokens, heads, d] normed (weight None: not) and turned at positions [axes, tokens]; the result, and what
    its bound is made of: the size of each element's pair before the turn."""
    y = x.astype(np.float64)
    if weight is not None:
        y = y / np.sqrt((y ** 2).mean(-1, keepdims=True) + eps) * (weight + offset)
    z, size = y.copy(), np.abs(y)
    h = len(freq)
    for i in range(h):
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
        # the angle modulo a turn, in whole numbers: positions up to 2^31 lose nothing
        turns = round(freq[i] / (2 * math.pi) * 2.0 ** 64)
        a = np.array([(int(t) * turns) % (1 << 64) / 2.0 ** 64 for t in positions[axis[i]]])[:, None] * 2 * math.pi
        c, s = np.cos(a), np.sin(a)
        z[..., p], z[..., q] = y[..., p] * c - y[..., q] * s, y[..., p] * s + y[..., q] * c
        size[..., p] = size[..., q] = np.abs(y[..., p]) + np.abs(y[..., q])
    return z, size


def turn_bound(z, size, d, dtype):
    """The mean of squares is a sum of d products (each rounding 2^-24, in any order, half of it in the root); root,
    division, weight and its offset add 6 units of 2^-24. An angle of up to half a turn is off by 2^-25 of its 1 in
    units of half a turn (pi 2^-25 < 2^-23) and sine and cosine by 2 units of 2^-24, so that an element of the pair
    is off by under 2^-22 of the pair's sum, and its two products and sum round 2 more units. One rounding at the end
    (fp16: to steps of 2^-24 at least)."""
    return UNIT[dtype] * np.abs(z) + size * ((d / 2 + 8) * 2.0 ** -24 + 2.0 ** -21) + \
        (2.0 ** -25 if dtype == "f16" else 1e-38)


def prompt_attention(k, v, table, lengths, slots, cu, q, scale):
    """out, lse of packed causal prompts, and a bound's ingredients (as tests.kv_ref.attention)."""
    total, Hq, d = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    out, lse = np.zeros((total, Hq, d)), np.full((total, Hq), -np.inf)
    mag, smag = np.zeros((total, Hq, d)), np.zeros((total, Hq))
    for b, slot in enumerate(slots):
        n = cu[b + 1] - cu[b]
        if slot < 0 or n == 0:
            continue
        L = int(lengths[slot])
        for h in range(Hkv):
            kc, vc = entries(k, table, slot, h, L), entries(v, table, slot, h, L)
            for j in range(n):
                keys, vals = kc[:L - n + j + 1], vc[:L - n + j + 1]
                for x in range(h * G, (h + 1) * G):
                    r = cu[b] + j
                    s = keys @ q[r, x] * scale
                    m = s.max()
                    e = np.exp(s - m)
                    lse[r, x] = m + math.log(e.sum())
                    p = e / e.sum()
                    out[r, x], mag[r, x] = p @ vals, p @ np.abs(vals)
                    smag[r, x] = (np.abs(keys) @ np.abs(q[r, x])).max() * abs(scale)
    return out, lse, mag, smag


class Prompt:
    """A cache and packed prompts [(rows, entries before them)]. Entries past a length, pages that nobody holds and
    rows of no sequence are NaN. written: the prompts' own entries are in the cache already; blank: no entry's key and value is."""

    def __init__(self, seed, dtype, prompts, Hq, Hkv, d, page, kind="heads", pad=(), gap=0, spread=1.0, written=True,
                 q_kind="plain", blank=False):
        from hybrid_ssm_gated_gb300 import kv

        self.kv, r = kv, np.random.default_rng(seed)
        self.r, self.dtype, self.Hq, self.Hkv, self.d, self.page = r, dtype, Hq, Hkv, d, page
        B = self.B = len(prompts)
        self.prompts = prompts
        ns = [n for n, _ in prompts]
        self.cu = np.concatenate([[gap], gap + np.cumsum(ns)]).astype(np.int32)
        self.total = int(self.cu[-1]) + gap
        lens = [n + p for n, p in prompts]
        need = [-(-n // page) for n in lens]
        num_slots, num_pages, max_pages = B + 2, sum(need) + 2, max(need + [1]) + 1
        self.slots = r.permutation(num_slots)[:B].astype(np.int32)
        order, at = r.permutation(num_pages), 0
        self.table = np.full((num_slots, max_pages), -7, np.int32)
        self.lengths = np.zeros(num_slots, np.int32)
        for b in range(B):
            self.table[self.slots[b], :need[b]] = order[at:at + need[b]]
            at += need[b]
            self.lengths[self.slots[b]] = lens[b] if written else prompts[b][1]
        self.counts = self.lengths + 11
        for b in pad:
            self.slots[b] = -1
        # values as the cache's type holds them, on the host first (one copy for each pool)
        dt = TORCH[dtype]
        k0, v0 = (torch.full((num_pages, Hkv, page, d), float("nan"), dtype=dt) for _ in range(2))
        for b in range(B):
            if self.slots[b] >= 0 and not blank:
                L = lens[b] if written else prompts[b][1]
                for pool, s in ((k0, spread), (v0, 1.0)):
                    x = torch.from_numpy(r.normal(size=(L, Hkv, d)) * s).to(dt)
                    for j in range(-(-L // page)):
                        part = x[j * page:(j + 1) * page]
                        pool[int(self.table[self.slots[b], j]), :, :part.shape[0]] = part.transpose(0, 1)
        self.k, self.v = layout((num_pages, Hkv, page, d), dtype, kind)
        self.k.copy_(k0), self.v.copy_(v0)
        rows = lambda H, s: torch.from_numpy(r.normal(size=(self.total, H, d)) * s).to(dt).cuda()
        self.q, self.kn, self.vn = rows(Hq, spread), rows(Hkv, spread), rows(Hkv, 1.0)
        for x in (self.q, self.kn, self.vn):
            x[:gap] = float("nan")
            x[int(self.cu[-1]):] = float("nan")
        if q_kind == "joint":  # parts of one projection's output
            x = torch.cat([self.q, self.kn, self.vn], 1)
            self.q, self.kn, self.vn = x.split([Hq, Hkv, Hkv], 1)
        elif q_kind == "odd":  # rows off the 16-byte grid
            def odd(t):
                y = torch.empty(*t.shape[:2], d + 1, dtype=dt, device="cuda")[..., 1:]
                return y.copy_(t)
            self.q, self.kn, self.vn = odd(self.q), odd(self.kn), odd(self.vn)
        shape = (num_pages, Hkv, page)
        self.weights = torch.from_numpy(r.exponential(size=shape)).float().cuda()
        self.stamps = torch.from_numpy(r.integers(0, 9, size=shape)).int().cuda()
        self.scale = 1.0 / math.sqrt(d)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.sync()

    def sync(self):
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
        self.d_slots, self.d_cu = dev(self.slots), dev(self.cu)
        self.d_lengths, self.d_counts, self.d_table = dev(self.lengths), dev(self.counts), dev(self.table)
        self.cache = self.kv.KVCache(self.k, self.v, self.d_table, self.d_lengths, self.d_counts, self.weights,
                                     self.stamps)

    def attend(self, stream=None, with_lse=True, fill=0xFF):
        guards = []
        out = guarded(self.q.shape, self.q.dtype, guards).fill_(7.0)
        lse = guarded(self.q.shape[:2], torch.float32, guards).fill_(7.0) if with_lse else None
        ws = guarded((self.kv.kv_prompt_workspace(self.cache, self.B, self.q).numel(),), torch.uint8, guards).fill_(fill)
        torch.cuda.synchronize()
        self.kv.kv_prompt_attention(self.cache, self.d_slots, self.d_cu, self.q, out, self.err, ws, lse=lse,
                                    scale=self.scale, stream=stream)
        torch.cuda.synchronize()
        assert canaries_intact(guards)
        return out, lse

    def owned(self):
        """Which rows are some sequence's."""
        x = np.zeros(self.total, bool)
        for b in range(self.B):
            x[self.cu[b]:self.cu[b + 1]] = True
        return x

    def compare(self, out, lse, ref, rl, mag, smag, rows):
        o, z = host(out)[rows], host(lse)[rows]
        bad = ~(np.abs(o - ref[rows]) <= out_bound(mag, smag, self.d, self.dtype)[rows])
        assert not bad.any(), f"{bad.sum()} outputs off, by {np.nanmax(np.abs(o - ref[rows])):.3e}, rows " \
                              f"{np.unique(np.nonzero(bad)[0])[:8]}"
        assert np.array_equal(np.isneginf(z), np.isneginf(rl[rows]))
        fin = np.isfinite(rl[rows])
        off = np.abs(z[fin] - rl[rows][fin])
        assert (off <= lse_bound(rl, smag, self.d)[rows][fin]).all(), f"lse off by {off.max():.3e}"

    def check(self, expect_err=0):
        out, lse = self.attend()
        assert int(self.err.item()) == expect_err
        ref = prompt_attention(host(self.k), host(self.v), self.table, self.lengths, self.slots, self.cu, host(self.q),
                               self.scale)
        own = self.owned()
        self.compare(out, lse, *ref, own)
        assert (out[~own] == 7.0).all() and (lse[~own] == 7.0).all()  # rows of no sequence are left as they were
        return out, lse
