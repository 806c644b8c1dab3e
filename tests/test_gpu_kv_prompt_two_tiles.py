"""Unusual scores in every form of the prompt attention: few heads (one tile of rows a unit), and as many heads as give each
SM a unit of two tiles."""
import math

import numpy as np
import pytest
import torch

from hybrid_ssm_gated_gb300 import build, kv
from tests.kv_ref import UNIT, host, lse_bound, out_bound
from tests.prompt_ref import Prompt
from tests.test_gpu_kv_prompt import check_sampled

pytestmark = pytest.mark.gpu

DTYPES = ["bf16", "f16", "f32"]
FEW, MANY = (4, 2), (80 * 8, 80)  # query and key heads


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    kv.lib()


def make(seed, dtype, heads, prompts=((90, 45), (50, 0)), d=64, **kw):
    total = sum(n for n, _ in prompts)
    if heads == MANY and dtype != "f32":  # (units of two tiles for every SM, and more than sequences)
        units = total // (2 * (128 // 8))
        assert units * 80 >= 152 and units >= len(prompts)
    return Prompt(seed, dtype, list(prompts), Hq=heads[0], Hkv=heads[1], d=d, page=16, **kw)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scale", [0.0, -0.3, -1e-30, 3.0])
@pytest.mark.parametrize("d", [64, 128])
def test_scales(dtype, scale, d):
    c = make(90, dtype, MANY, d=d)
    c.scale = scale
    check_sampled(c, 13)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("spread", [30.0, 1000.0])
def test_scores_far_apart(dtype, spread):
    check_sampled(make(91, dtype, MANY, spread=min(spread, 60.0) if dtype == "f16" else spread), 13)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads,prompts", [(MANY, [(150, 140)]), (FEW, [(40, 9000)])], ids=["two tiles", "joined"])
def test_scores_beyond_2_24(dtype, heads, prompts):
    """Equal scores of 2^30 in a row: weights are equal whatever the reference is rounded to, in a block and where the
    parts of several are joined."""
    c = make(92, dtype, heads, prompts)
    n, p = prompts[0]
    c.k.fill_(64.0), c.q.fill_(64.0)
    c.v.copy_(torch.arange(c.page, device="cuda").view(1, 1, -1, 1).expand_as(c.v) % 2)
    c.scale = 2.0 ** 12
    out, _ = c.attend()
    assert int(c.err.item()) == 0
    seen = p + 1 + np.arange(n)
    want = (seen // 2) / seen
    # weights of 1 and their sums are exact; tensor memory cuts off 2^-21 of a sum at most for each product of 16 keys
    assert np.abs(host(out) - want[:, None, None]).max() <= 2.0 ** -19 + UNIT[dtype] + (p + n) / 16 * 2.0 ** -21


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads", [FEW, MANY], ids=["one tile", "two tiles"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("e", [20, 95], ids=["in the prefix", "of row 50"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_keys_that_are_not_finite(dtype, heads, d, e, bad):
    """A NaN key makes every row that sees it NaN, and so does an infinite score; a score of -infinity takes its entry out of
    the row. Rows that do not see it, and those of other heads and sequences, are the same to the bit."""
    first = max(0, e - 45)  # the first row that sees it
    c, want = make(93, dtype, heads, d=d), make(93, dtype, heads, d=d)
    slot, G = c.slots[0], heads[0] // heads[1]
    c.k[int(c.table[slot, e // 16]), 1, e % 16, 3] = bad
    got, lse = c.attend()
    base, base_lse = want.attend()
    hit = torch.zeros_like(lse, dtype=torch.bool)
    hit[first:90, G:2 * G] = True
    assert torch.equal(got[~hit], base[~hit]) and torch.equal(lse[~hit], base_lse[~hit])
    sign = torch.sign(c.q[..., 3].float()) * (1.0 if bad > 0 else -1.0)
    gone = hit & (sign < 0) if not math.isnan(bad) else torch.zeros_like(hit)
    lost = hit & ~gone
    assert got[lost].isnan().all() and lse[lost].isnan().all()
    if not gone.any():
        return
    # rows without the entry, by the definition in 64 bits
    pages = torch.from_numpy(c.table[slot, :-(-135 // 16)]).long().cuda()
    k, v = (x[pages, 1].reshape(-1, d)[:135].double() for x in (want.k, want.v))
    s = torch.einsum("nhd,ed->nhe", c.q[:90, G:2 * G].double(), k) * c.scale
    seen = torch.arange(135, device="cuda") <= 45 + torch.arange(90, device="cuda")[:, None]
    seen[:, e] = False
    s = s.masked_fill(~seen[:, None], float("-inf"))
    w, z = torch.softmax(s, -1), torch.logsumexp(s, -1)
    smag = torch.einsum("nhd,ed->nhe", c.q[:90, G:2 * G].double().abs(), k.abs()).amax(-1) * c.scale
    o, mag, z, smag, pick = (host(x) for x in (w @ v, w @ v.abs(), z, smag, gone[:90, G:2 * G]))
    assert (np.abs(host(got[:90, G:2 * G]) - o) <= out_bound(mag, smag, d, dtype))[pick].all()
    assert (np.abs(host(lse[:90, G:2 * G]) - z) <= lse_bound(z, smag, d))[pick].all()
