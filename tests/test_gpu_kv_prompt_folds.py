"""Prompt attention whose blocks take long runs of one unit's keys: sums that the tensor-core kernel folds several times,
over values that are not all alike, while the rows' largest scores rise before, between and behind the folds. All the
sequences of a call name one slot: attention writes nothing, so a slot may stand in a call more than once."""
import math

import numpy as np
import pytest
import torch

from hybrid_ssm_gated_gb300 import build, kv
from tests.kv_ref import TORCH, host, lse_bound, out_bound

pytestmark = pytest.mark.gpu

B, PAGE, RISE = 160, 64, 10.0  # sequences (more units than SMs); entries of a page; powers of two that a step rises by
FOLD = {"bf16": 16384, "f16": 4096}  # entries of a sum in tensor memory


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    kv.lib()


class Rising:
    """B sequences of n rows over one cache of L entries, whose keys lean along every query in `steps` steps: the scores
    rise by RISE powers of two at each, and the values fall (by 18 powers in all), so that earlier steps still show."""

    def __init__(self, dtype, d, n, L, steps):
        g = torch.Generator(device="cuda").manual_seed(d + L)
        rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)
        dt, self.dtype, self.d, self.n, self.L = TORCH[dtype], dtype, d, n, L
        pages = -(-L // PAGE)
        entry = torch.arange(pages * PAGE, device="cuda")
        level = sum(((entry >= x).float() for x in steps), torch.zeros(pages * PAGE, device="cuda"))
        k, v = rnd(pages * PAGE, d), rnd(pages * PAGE, d)
        k[:, 0] = level * RISE * math.log(2.0) * math.sqrt(d) / 8
        v *= torch.exp2(9.0 - 18.0 / max(1, len(steps)) * level)[:, None]
        k[L:], v[L:] = float("nan"), float("nan")
        self.k, self.v = k.to(dt), v.to(dt)
        q = rnd(B * n, 1, d)
        q[..., 0] = 8.0
        self.q = q.to(dt)
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(L)).int()
        pool = lambda x: torch.empty(pages, 1, PAGE, d, dtype=dt, device="cuda").index_copy_(
            0, order.long().cuda(), x.view(pages, 1, PAGE, d))
        i32 = lambda x: torch.as_tensor(x, dtype=torch.int32).cuda()
        self.cache = kv.KVCache(pool(self.k), pool(self.v), order.view(1, -1).cuda(), i32([L]))
        self.slots, self.cu, self.err = i32([0] * B), i32(np.arange(B + 1) * n), i32([0])

    def attend(self):
        out, lse = torch.full_like(self.q, 7.0), torch.full((B * self.n, 1), 7.0, device="cuda")
        kv.kv_prompt_attention(self.cache, self.slots, self.cu, self.q, out, self.err,
                               kv.kv_prompt_workspace(self.cache, B, self.q), lse=lse)
        assert int(self.err.item()) == 0
        return host(out)[:, 0], host(lse)[:, 0]

    def exact(self, rows):
        """The last row's scores (in 64 bits), and outputs, log-sum-exps and the bounds' ingredients of `rows`."""
        k, v, q = self.k[:self.L].double(), self.v[:self.L].double(), self.q[rows, 0].double()
        s = q @ k.T / math.sqrt(self.d)
        last = self.L - self.n + torch.as_tensor(rows, device="cuda") % self.n
        s.masked_fill_(torch.arange(self.L, device="cuda") > last[:, None], float("-inf"))
        w = torch.softmax(s, -1)
        smag = (q.abs() @ k.abs().T).amax(-1) / math.sqrt(self.d)
        return s[-1], w @ v, torch.logsumexp(s, -1), w @ v.abs(), smag


def bounds(c, z, mag, smag):
    """As tests.kv_ref's, and what tensor memory cuts off: 2^-21 of a sum at most for each product of 16 keys of a fold."""
    cut = FOLD[c.dtype] / 16 * 2.0 ** -21 if c.dtype in FOLD else 0.0
    return out_bound(mag, smag, c.d, c.dtype) + mag * cut, lse_bound(z, smag, c.d)


CASES = [("bf16", 64, 256, 60000), ("bf16", 128, 256, 60000), ("bf16", 256, 128, 60000),
         ("f16", 64, 256, 20000), ("f16", 128, 256, 20000), ("f16", 256, 128, 20000), ("f32", 64, 64, 20000)]


@pytest.mark.parametrize("dtype,d,n,L", CASES)
@pytest.mark.parametrize("steps", [6, 25])
def test_folds_while_the_reference_rises(dtype, d, n, L, steps):
    """A block takes about one unit's keys (B units over 152 SMs): 3.6 folds of bf16 and 4.9 of fp16 from a unit's
    beginning, fewer where a range begins later, so that every step lies behind some fold and before another."""
    edges = [round(L * (i + 0.6) / (steps + 0.3)) for i in range(steps)]
    c = Rising(dtype, d, n, L, edges)
    out, lse = c.attend()
    rows = np.unique(np.concatenate([np.arange(0, B * n, n), np.arange(n - 1, B * n, n), np.arange(0, B * n, 89)]))
    x, o, z, mag, smag = (x.cpu().numpy() for x in c.exact(rows))
    ob, zb = bounds(c, z, mag, smag)
    off = np.abs(out[rows] - o)
    assert (off <= ob).all(), f"{(off > ob).sum()} outputs off, by {(off / ob).max():.2f} bounds"
    assert (np.abs(lse[rows] - z) <= zb).all(), f"lse off by {np.abs(lse[rows] - z).max():.3e}"
    if dtype == "f32":
        return
    # what the bounds are for: folds that are added up without their factor, by the definition in 64 bits, miss them
    f, e = FOLD[dtype], c.v[:L].double().cpu().numpy()
    parts = [x[i:i + f] for i in range(0, L, f)]
    refs = np.maximum.accumulate([p.max() for p in parts])
    sums = [np.exp(p - m) @ e[i * f:i * f + len(p)] for i, (p, m) in enumerate(zip(parts, refs))]
    wrong = sum(sums) / np.exp(x - refs[-1]).sum()
    assert (np.abs(wrong - o[-1]) > 10 * ob[-1]).any()


@pytest.mark.parametrize("dtype,d,n,L", CASES)
def test_folds_without_a_rise(dtype, d, n, L):
    """Values of both signs under scores of one size."""
    c = Rising(dtype, d, n, L, [])
    out, lse = c.attend()
    rows = np.unique(np.concatenate([np.arange(0, B * n, n), np.arange(n - 1, B * n, n)]))
    _, o, z, mag, smag = (x.cpu().numpy() for x in c.exact(rows))
    ob, zb = bounds(c, z, mag, smag)
    off = np.abs(out[rows] - o)
    assert (off <= ob).all(), f"{(off > ob).sum()} outputs off, by {(off / ob).max():.2f} bounds"
    assert (np.abs(lse[rows] - z) <= zb).all(), f"lse off by {np.abs(lse[rows] - z).max():.3e}"
