"""GPU parity of the prompt operators of include/kv.h against their definitions in 64 bits
(tests/prompt_ref.py): causal attention of packed prompts over the cache, norms and rotations, appends.
Bounds are derived beside the references."""
import math

import numpy as np
import pytest
import torch

from hybrid_ssm_gated_gb300 import build, gdn, kv
from tests import prompt_ref as ref
from tests.gpu_util import canaries_intact, guarded
from tests.kv_ref import TORCH, UNIT, host
from tests.prompt_ref import Prompt

pytestmark = pytest.mark.gpu

DTYPES = ["bf16", "f16", "f32"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    kv.lib()


# ---------------------------------------------------------------- attention

PROMPTS = [[(1, 0)], [(1, 5), (0, 9), (2, 0), (3, 130)], [(15, 0), (16, 1), (17, 0)], [(63, 2), (64, 64), (65, 0)],
           [(127, 0), (128, 128), (129, 7)], [(300, 0), (1, 300), (33, 250)]]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("prompts", PROMPTS, ids=str)
@pytest.mark.parametrize("d,page", [(64, 16), (128, 16), (256, 32)])
def test_lengths(dtype, prompts, d, page):
    Prompt(1, dtype, prompts, Hq=4, Hkv=2, d=d, page=page).check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("G", [1, 3, 5, 8, 16, 71, 128, 160])
@pytest.mark.parametrize("d", [64, 256])
def test_heads_a_group(dtype, G, d):
    """Groups that a block of rows holds whole, that it cuts, and that are larger than it."""
    n = 3 if G > 16 else 70
    Prompt(2, dtype, [(n, 40), (n + 1, 0)], Hq=2 * G, Hkv=2, d=d, page=16).check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [8, 40, 72, 80, 96, 120, 136, 192, 200])
def test_head_sizes(dtype, d):
    Prompt(3, dtype, [(133, 0), (40, 100)], Hq=6, Hkv=3, d=d, page=16).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [1, 3, 7, 33, 129, 255])
def test_head_sizes_off_the_grid(dtype, d):
    Prompt(4, dtype, [(66, 3), (5, 0)], Hq=4, Hkv=2, d=d, page=8).check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("page", [1, 5, 8, 24, 48, 64, 100, 128, 256])
def test_page_sizes(dtype, page):
    Prompt(5, dtype, [(200, 100), (131, 0), (7, 9)], Hq=4, Hkv=2, d=64, page=page).check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["heads", "places", "joint", "odd"])
@pytest.mark.parametrize("q_kind", ["plain", "joint", "odd"])
def test_layouts(dtype, kind, q_kind):
    Prompt(6, dtype, [(150, 10), (33, 0)], Hq=4, Hkv=2, d=64, page=16, kind=kind, q_kind=q_kind).check()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,G", [(128, 4), (256, 8), (64, 3)])
def test_few_rows_over_a_long_cache(dtype, d, G):
    """Units that many blocks of the grid share, and whose sums are folded more than once."""
    Prompt(7, dtype, [(3, 20000), (40, 7000)], Hq=G, Hkv=1, d=d, page=64).check()


def check_sampled(c, step, more=()):
    """Every step-th row and `more` against the definition in 64 bits, formed on the device."""
    out, lse = c.attend()
    assert int(c.err.item()) == 0
    k, v, q, G = c.k.double(), c.v.double(), c.q.double(), c.Hq // c.Hkv
    rows = np.unique(np.concatenate([np.arange(0, c.total, step), c.cu[1:] - 1, c.cu[:-1], more])).astype(int)
    for b, (n, p) in enumerate(c.prompts):
        if n == 0 or c.slots[b] < 0:
            continue
        pages = torch.from_numpy(c.table[c.slots[b], :-(-(n + p) // c.page)]).long().cuda()
        kc, vc = (x[pages].transpose(0, 1).reshape(c.Hkv, -1, c.d)[:, :n + p] for x in (k, v))
        for r in rows[(rows >= c.cu[b]) & (rows < c.cu[b + 1])]:
            L = p + int(r) - int(c.cu[b]) + 1
            qr = q[r].view(c.Hkv, G, c.d)
            s = qr @ kc[:, :L].transpose(1, 2) * c.scale
            w = torch.softmax(s, -1)
            want, mag = (w @ vc[:, :L]).cpu().numpy(), (w @ vc[:, :L].abs()).cpu().numpy()
            smag = ((qr.abs() @ kc[:, :L].abs().transpose(1, 2)).amax(-1) * abs(c.scale)).cpu().numpy()
            assert (np.abs(host(out[r]).reshape(want.shape) - want) <= ref.out_bound(mag, smag, c.d, c.dtype)).all(), r
            z = torch.logsumexp(s, -1).cpu().numpy()
            assert (np.abs(host(lse[r]).reshape(z.shape) - z) <= ref.lse_bound(z, smag, c.d)).all(), r
    return out, lse


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_long_prompts(dtype, d):
    """Several units a key head, cut by the ranges of the grid; every 37th row is compared."""
    check_sampled(Prompt(8, dtype, [(2100, 0), (1500, 3000)], Hq=4, Hkv=2, d=d, page=64), 37)


# (rows, entries before them), query and key heads: units for every SM, so that each holds two tiles of rows
MANY_UNITS = [([(2500, 0)], 16, 2), ([(300, 20), (0, 5), (411, 900), (63, 0)], 64, 8), ([(1, 0), (1000, 130)], 40, 8),
              ([(1800, 3000)], 24, 24), ([(640, 0), (33, 1)], 96, 8), ([(290, 77)], 71 * 2, 2), ([(160, 7000)], 128 * 2, 2)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 80, 128])
@pytest.mark.parametrize("prompts,Hq,Hkv", MANY_UNITS, ids=str)
def test_many_units(dtype, d, prompts, Hq, Hkv):
    total = sum(n for n, _ in prompts)
    assert total // (2 * (128 // (Hq // Hkv))) * Hkv >= 152
    check_sampled(Prompt(27, dtype, prompts, Hq=Hq, Hkv=Hkv, d=d, page=16), max(1, total // 60))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("leader", [False, True])
@pytest.mark.parametrize("heads", [1, 160])
def test_sums_of_a_long_cache_do_not_shrink(dtype, d, leader, heads):
    """Every value is 1 and so is every output: equal weights, or one entry that holds most of the weight. A sum of
    weights that lost more than half a unit of rounding of the cache's type would not come out as 1."""
    n, p = (140, 60000) if heads == 1 else (260, 20000)
    c = Prompt(9, dtype, [(n, p)], Hq=heads, Hkv=heads, d=d, page=64, blank=True)
    c.k.zero_()
    c.v.fill_(1.0)
    c.q.fill_(1.0)
    if leader:
        c.k[int(c.table[c.slots[0], 0]), :, 0] = 10.0 / math.sqrt(d)
    out, _ = c.attend()
    assert int(c.err.item()) == 0
    assert (out.float() - 1.0).abs().max().item() <= UNIT[dtype]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("heads", [(4, 2), (80 * 8, 80)], ids=str)
def test_values_that_are_not_finite_reach_only_rows_that_see_them(dtype, d, bad, heads):
    Hq, Hkv = heads
    c = Prompt(10, dtype, [(90, 45), (20, 0)], Hq=Hq, Hkv=Hkv, d=d, page=16)
    slot, e = c.slots[0], 45 + 50  # the entry of row 50
    c.v[int(c.table[slot, e // 16]), 1, e % 16, 3] = bad
    want = Prompt(10, dtype, [(90, 45), (20, 0)], Hq=Hq, Hkv=Hkv, d=d, page=16)
    got, base = c.attend()[0], want.attend()[0]
    hit = torch.zeros_like(got, dtype=torch.bool)
    hit[50:90, Hq // Hkv:2 * (Hq // Hkv), 3] = True
    assert torch.equal(got[~hit], base[~hit])
    assert not got[hit].isfinite().any() and (math.isnan(bad) or (got[hit] == bad).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_keys_that_are_not_finite_reach_only_rows_that_see_them(dtype, bad):
    make = lambda: Prompt(11, dtype, [(90, 45), (20, 0)], Hq=4, Hkv=2, d=64, page=16)
    c, want = make(), make()
    e = 45 + 50
    c.k[int(c.table[c.slots[0], e // 16]), 1, e % 16, 3] = bad
    got, base = c.attend()[0], want.attend()[0]
    hit = torch.zeros_like(got, dtype=torch.bool)
    hit[50:90, 2:] = True
    assert torch.equal(got[~hit], base[~hit])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("spread", [30.0, 1000.0])
def test_scores_far_apart(dtype, spread):
    """Scores of up to 10^5 and more: one entry holds all of a row's weight."""
    if dtype == "f16":
        spread = min(spread, 60.0)
    c = Prompt(12, dtype, [(140, 20)], Hq=4, Hkv=2, d=64, page=16, spread=spread)
    c.check()


@pytest.mark.parametrize("dtype", DTYPES)
def test_scores_beyond_2_24(dtype):
    """Equal scores of 2^30 in a row: weights are equal whatever the reference is rounded to."""
    c = Prompt(13, dtype, [(150, 140)], Hq=2, Hkv=1, d=64, page=16)
    c.k.fill_(64.0), c.q.fill_(64.0)
    c.v.copy_(torch.arange(c.page, device="cuda").view(1, 1, -1, 1).expand_as(c.v) % 2)
    c.scale = 2.0 ** 12
    out, _ = c.attend()
    seen = np.arange(141, 291)
    want = (seen // 2) / seen
    assert np.abs(host(out)[..., 0] - want[:, None]).max() <= 2.0 ** -19 + UNIT[dtype]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scale", [0.0, -0.3])
def test_scales(dtype, scale):
    c = Prompt(14, dtype, [(80, 60), (129, 0)], Hq=4, Hkv=2, d=64, page=16)
    c.scale = scale
    c.check()


@pytest.mark.parametrize("dtype", DTYPES)
def test_padding_and_rows_of_no_sequence(dtype):
    c = Prompt(15, dtype, [(40, 3), (50, 0), (70, 9)], Hq=4, Hkv=2, d=64, page=16, pad=(1,), gap=5)
    out, lse = c.check()
    assert (out[45:95] == 0).all() and torch.isneginf(lse[45:95]).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("what,bit", [("slot", gdn.DEVERR_SLOT), ("short", kv.DEVERR_LENGTH), ("negative", kv.DEVERR_LENGTH),
                                      ("long", kv.DEVERR_LENGTH)])
def test_refused_sequences(dtype, what, bit):
    c = Prompt(16, dtype, [(40, 3), (50, 0), (70, 9)], Hq=4, Hkv=2, d=64, page=16)
    if what == "slot":
        c.slots[1] = len(c.lengths)
    else:
        c.lengths[c.slots[1]] = {"short": 49, "negative": -1, "long": c.table.shape[1] * 16 + 1}[what]
    slots = c.slots.copy()
    c.sync()
    out, lse = c.attend()
    assert int(c.err.item()) == bit
    slots[1] = -1  # (how the others' keys are split may change with it: they are compared with the definition)
    own = np.r_[0:40, 90:160]
    c.compare(out, lse, *ref.prompt_attention(host(c.k), host(c.v), c.table, c.lengths, slots, c.cu, host(c.q), c.scale), own)
    assert (out[40:90] == 0).all() and torch.isneginf(lse[40:90]).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("page", [-7, 10 ** 6])
@pytest.mark.parametrize("heads", [(4, 2), (25 * 8, 25)], ids=str)
def test_a_page_outside_the_pool(dtype, page, heads):
    """A page in the middle of the second sequence: blocks that reach it are refused, the others and other sequences
    are right."""
    c = Prompt(17, dtype, [(40, 3), (300, 20), (70, 9)], Hq=heads[0], Hkv=heads[1], d=64, page=16)
    want, wl = c.attend()
    c.table[c.slots[1], 14] = page
    c.sync()
    out, lse = c.attend()
    assert int(c.err.item()) == kv.DEVERR_PAGE
    own = np.r_[0:40, 340:410]
    assert torch.equal(out[own], want[own]) and torch.equal(lse[own], wl[own])
    same = (out == want).all(2) & (lse == wl)
    zero = (out == 0).all(2) & torch.isneginf(lse)
    assert (same | zero)[40:340].all() and zero[40 + 14 * 16 - 20:340].all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_offsets_out_of_order(dtype):
    c = Prompt(18, dtype, [(40, 3), (50, 0), (70, 9)], Hq=4, Hkv=2, d=64, page=16)
    want = ref.prompt_attention(host(c.k), host(c.v), c.table, c.lengths, c.slots, c.cu, host(c.q), c.scale)
    c.cu = np.array([0, 40, 30, 161], np.int32)  # the second decreases, the third passes the rows
    c.sync()
    out, lse = c.attend()
    assert int(c.err.item()) == gdn.DEVERR_SEQLEN
    c.compare(out, lse, *want, np.r_[0:40])
    assert (out[40:] == 7.0).all() and (lse[40:] == 7.0).all()


def test_offsets_negative():
    c = Prompt(18, "bf16", [(40, 3), (50, 0)], Hq=4, Hkv=2, d=64, page=16)
    c.cu = np.array([-5, 40, 90], np.int32)
    c.sync()
    out, _ = c.attend()
    assert int(c.err.item()) == gdn.DEVERR_SEQLEN and (out[:40] == 7.0).all() and (out[40:] != 7.0).any()


@pytest.mark.parametrize("dtype", DTYPES)
def test_no_rows_at_all(dtype):
    c = Prompt(19, dtype, [(0, 3), (0, 0)], Hq=4, Hkv=2, d=64, page=16, gap=4)
    out, lse = c.attend()
    assert int(c.err.item()) == 0 and (out == 7.0).all() and (lse == 7.0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B", [40, 700])
def test_many_sequences(dtype, B):
    """More sequences than a block has threads."""
    r = np.random.default_rng(20)
    Prompt(20, dtype, [(int(r.integers(0, 4)), int(r.integers(0, 20))) for _ in range(B)], Hq=2, Hkv=1, d=64, page=8).check()


@pytest.mark.parametrize("dtype", DTYPES)
def test_the_same_call_gives_the_same_bits(dtype):
    c = Prompt(21, dtype, [(500, 3000), (100, 0)], Hq=8, Hkv=2, d=128, page=16)
    a, la = c.attend()
    b, lb = c.attend(fill=1)
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_without_lse_and_on_another_stream():
    c = Prompt(22, "bf16", [(300, 100), (20, 0)], Hq=4, Hkv=2, d=128, page=16)
    want, _ = c.attend()
    s = torch.cuda.Stream()
    out, _ = c.attend(stream=s, with_lse=False)
    assert torch.equal(out, want)


def test_two_calls_at_once():
    """On two streams, with a workspace each."""
    cs = [Prompt(23 + i, "bf16", [(700, 2000), (50, 0)], Hq=8, Hkv=2, d=128, page=16) for i in range(2)]
    want = [c.attend()[0] for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    got = [torch.empty_like(c.q) for c in cs]
    ws = [kv.kv_prompt_workspace(c.cache, c.B, c.q) for c in cs]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s, o, w in zip(cs, streams, got, ws):
            kv.kv_prompt_attention(c.cache, c.d_slots, c.d_cu, c.q, o, c.err, w, scale=c.scale, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_and_replayed_with_other_lengths(dtype):
    """A graph of an append and the attention behind it; each replay takes the lengths as they are then."""
    c = Prompt(25, dtype, [(60, 0), (30, 0)], Hq=4, Hkv=2, d=64, page=16, written=False)
    c.table[c.slots[0], :] = np.arange(c.table.shape[1])
    c.table = np.full((c.table.shape[0], 16), -1, np.int32)
    pages = np.random.default_rng(1).permutation(32)
    c.table[c.slots[0]], c.table[c.slots[1]] = pages[:16], pages[16:]
    c.k, c.v = (torch.full((32, 2, 16, 64), float("nan"), dtype=TORCH[dtype], device="cuda") for _ in range(2))
    c.weights, c.stamps = torch.ones(32, 2, 16, device="cuda"), torch.zeros(32, 2, 16, dtype=torch.int32, device="cuda")
    c.sync()
    rot = kv.Rotary(10000.0 ** (-torch.arange(32) / 32.0))
    out, lse, qt = torch.empty_like(c.q), torch.empty(c.total, 4, device="cuda"), torch.empty_like(c.q)
    ws = kv.kv_prompt_workspace(c.cache, 2, c.q)

    def call():
        kv.kv_append(c.cache, c.d_slots, c.d_cu, c.kn, c.vn, c.err, rotary=rot, q=c.q, q_out=qt)
        kv.kv_prompt_attention(c.cache, c.d_slots, c.d_cu, qt, out, c.err, ws, lse=lse, scale=c.scale)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for i in range(2, 4):
        g.replay()
        torch.cuda.synchronize()
        assert int(c.err.item()) == 0
        c.lengths[c.slots] = np.array([60, 30]) * i
        assert np.array_equal(c.d_lengths.cpu().numpy(), c.lengths)
        r = ref.prompt_attention(host(c.k), host(c.v), c.table, c.lengths, c.slots, c.cu, host(qt), c.scale)
        c.compare(out, lse, *r, c.owned())


def test_a_pool_past_4_gib():
    """Pages whose offsets pass 32 bits in elements and bytes."""
    Hkv, page, d = 2, 64, 128
    num = (1 << 32) // (Hkv * page * d) + 40
    k = torch.zeros(num, Hkv, page, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    small = Prompt(26, "bf16", [(150, 100)], Hq=4, Hkv=Hkv, d=d, page=page)
    want, wl = small.attend()
    table = torch.full((3, 5), -1, dtype=torch.int32)
    for j in range(4):
        src = int(small.table[small.slots[0], j])
        to = num - 1 - 3 * j
        k[to], v[to] = small.k[src], small.v[src]
        table[1, j] = to
    cache = kv.KVCache(k, v, table.cuda(), torch.tensor([0, 250, 0], dtype=torch.int32, device="cuda"),
                       torch.tensor([0, 250, 0], dtype=torch.int32, device="cuda"))
    slots = torch.tensor([1], dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(small.q), torch.empty_like(wl)
    kv.kv_prompt_attention(cache, slots, small.d_cu, small.q, out, small.err, kv.kv_prompt_workspace(cache, 1, small.q),
                           lse=lse)
    assert torch.equal(out, want) and torch.equal(lse, wl)
    # an append and a fork there
    cache.lengths[1] = 100
    kv.kv_append(cache, slots, small.d_cu, small.kn, small.vn, small.err)
    assert int(cache.lengths[1]) == 250 and torch.equal(k[num - 1 - 9, :, 249 - 192], small.kn[149])
    new = torch.full((1, 5), -1, dtype=torch.int32)
    new[0, 3] = num - 2
    kv.kv_fork(cache, slots, slots + 1, new.cuda(), small.err)
    assert torch.equal(v[num - 2, :, :58], v[num - 10, :, :58]) and cache.page_table[2, 3] == num - 2
    used = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv.kv_compact(cache, used, small.err, kv.kv_compact_workspace(cache))
    assert int(used) == 5 and int(cache.page_table[1:, :4].max()) == 4 and int(small.err) == 0
    kv.kv_prompt_attention(cache, slots + 1, small.d_cu, small.q, out, small.err, kv.kv_prompt_workspace(cache, 1, small.q),
                           lse=lse)
    assert int(small.err) == 0 and out.isfinite().all()


# ---------------------------------------------------------------- norm and rotation


def frequencies(rot):
    return [10000.0 ** (-2 * i / rot) for i in range(rot // 2)]


def check_rotate(dtype, B, T, Hq, Hkv, d, rot, axes=1, interleaved=False, norm="one", positions=None, in_place=False,
                 q_kind="plain", seed=30):
    r = np.random.default_rng(seed)
    dt = TORCH[dtype]
    rows = lambda H: torch.from_numpy(r.normal(size=(B, T, H, d)) * 3).to(dt).cuda()
    q, k = rows(Hq), rows(Hkv)
    if q_kind == "joint":
        q, k = torch.cat([q, k], 2).split([Hq, Hkv], 2)
    if q_kind == "odd":
        q, k = (torch.empty(*x.shape[:3], d + 1, dtype=dt, device="cuda")[..., 1:].copy_(x) for x in (q, k))
    w = {None: lambda H: None, "one": lambda H: r.normal(size=d), "heads": lambda H: r.normal(size=(H, d))}[norm]
    wq, wk = (x if x is None else x.astype(np.float32) for x in (w(Hq), w(Hkv)))
    f = frequencies(rot)
    axis = None if axes == 1 else [i % axes for i in range(rot // 2)]
    pos = r.integers(0, 5000, size=(axes, B, T)).astype(np.int32) if positions is None else positions
    dev = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()
    rot_ = kv.Rotary(f if rot else None, axis=axis, axes=axes, interleaved=interleaved, q_norm=dev(wq), k_norm=dev(wk),
                     eps=1e-5, offset=0.5)
    hq, hk = host(q).reshape(B * T, Hq, d), host(k).reshape(B * T, Hkv, d)
    guards = []
    qo = q if in_place else guarded(q.shape, dt, guards).fill_(7.0)
    ko = k if in_place else guarded(k.shape, dt, guards).fill_(7.0)
    kv.kv_norm_rotate(rot_, dev(pos) if rot else None, q=q, k=k, q_out=qo, k_out=ko)
    torch.cuda.synchronize()
    assert canaries_intact(guards)
    for x, o, weight in ((hq, qo, wq), (hk, ko, wk)):
        z, size = ref.turned(x, weight, 1e-5, 0.5, f, axis or [0] * len(f), pos.reshape(axes, -1), interleaved)
        off = np.abs(host(o).reshape(z.shape) - z)
        assert (off <= ref.turn_bound(z, size, d, dtype)).all(), f"off by {off.max():.3e}"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 128), (256, 256), (256, 64), (80, 40), (80, 20), (96, 24), (8, 8), (40, 0),
                                   (128, 16), (1, 0), (3, 2), (33, 32), (255, 254)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_sizes(dtype, d, rot, interleaved):
    check_rotate(dtype, 3, 5, 4, 2, d, rot, interleaved=interleaved)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("axes", [2, 3, 4])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_axes(dtype, axes, interleaved):
    check_rotate(dtype, 2, 33, 3, 1, 128, 96, axes=axes, interleaved=interleaved)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("norm", [None, "one", "heads"])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("q_kind", ["plain", "joint", "odd"])
def test_rotation_norms_and_strides(dtype, norm, in_place, q_kind):
    check_rotate(dtype, 2, 7, 5, 2, 64, 32, norm=norm, in_place=in_place, q_kind=q_kind)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rotation_of_many_tokens(dtype):
    check_rotate(dtype, 3, 5000, 2, 1, 64, 64)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_far_out(interleaved):
    """Positions up to the ends of their type: angles lose nothing."""
    pos = np.array([[[0, 1, -1, 2 ** 20 + 1, 10 ** 7 + 3, 2 ** 30 + 7, 2 ** 31 - 1, -2 ** 31]]], np.int32)
    check_rotate("f32", 1, 8, 2, 1, 128, 128, positions=pos, interleaved=interleaved)


def test_rotation_of_one_side():
    x = torch.randn(2, 3, 4, 64, device="cuda")
    rot = kv.Rotary(frequencies(64))
    pos = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    a, b = torch.empty_like(x), torch.empty_like(x)
    kv.kv_norm_rotate(rot, pos, q=x, q_out=a)
    kv.kv_norm_rotate(rot, pos, k=x, k_out=b)
    assert torch.equal(a, b) and not torch.equal(a, x)
    assert torch.equal(a[0, 0], x[0, 0])  # position 0


@pytest.mark.parametrize("dtype", DTYPES)
def test_rotation_of_zeros_and_odd_rows(dtype):
    """A row of zeros stays one; a row that is not finite reaches no other."""
    x = torch.randn(1, 4, 2, 64, device="cuda").to(TORCH[dtype])
    x[0, 1, 0] = 0
    y = x.clone()
    y[0, 2, 1, 5] = float("inf")
    rot = kv.Rotary(frequencies(64), q_norm=torch.ones(64, device="cuda"))
    pos = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
    a, b = torch.empty_like(x), torch.empty_like(x)
    kv.kv_norm_rotate(rot, pos, q=x, q_out=a)
    kv.kv_norm_rotate(rot, pos, q=y, q_out=b)
    assert (a[0, 1, 0] == 0).all()
    same = torch.ones(4, 2, dtype=torch.bool)
    same[2, 1] = False
    assert torch.equal(a[0][same], b[0][same])


# ---------------------------------------------------------------- append


def append_case(dtype, prompts, Hq=4, Hkv=2, d=64, page=16, rot=32, axes=1, norm=True, with_q=True, text=False, **kw):
    """Runs an append and compares everything it writes; what it must not write, bit for bit."""
    c = Prompt(40, dtype, prompts, Hq=Hq, Hkv=Hkv, d=d, page=page, written=False, **kw)
    r = c.r
    f, axis = frequencies(rot), [i % axes for i in range(rot // 2)]
    wq, wk = (r.normal(size=d).astype(np.float32) for _ in range(2))
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
    rotary = kv.Rotary(f, axis=axis, axes=axes, q_norm=dev(wq) if norm else None, k_norm=dev(wk) if norm else None,
                       eps=1e-5) if rot else None
    pos = r.integers(0, 3000, size=(axes, c.total)).astype(np.int32)
    guards = []
    qo = guarded(c.q.shape, c.q.dtype, guards).fill_(7.0) if with_q else None
    before = {n: host(getattr(c, n)) for n in ("k", "v", "weights", "stamps")}
    kv.kv_append(c.cache, c.d_slots, c.d_cu, c.kn, c.vn, c.err, rotary=rotary,
                 positions=None if text or not rot else dev(pos), q=c.q if with_q else None, q_out=qo)
    torch.cuda.synchronize()
    assert canaries_intact(guards)
    want, tol = {n: x.copy() for n, x in before.items()}, np.zeros(before["k"].shape)
    kn, vn = host(c.kn), host(c.vn)
    if text:
        for b, s in enumerate(c.slots):
            if s >= 0:
                pos[:, c.cu[b]:c.cu[b + 1]] = c.counts[s] + np.arange(c.cu[b + 1] - c.cu[b])
    if rot:
        kz, ks = ref.turned(kn, wk if norm else None, 1e-5, 0.0, f, axis, pos, False)
        bound = ref.turn_bound(kz, ks, d, dtype)
    else:
        kz, bound = kn, np.zeros(kn.shape)
    lengths, counts = c.lengths.copy(), c.counts.copy()
    for b, s in enumerate(c.slots):
        for j in range(c.cu[b + 1] - c.cu[b]):
            if s < 0:
                continue
            e, row = c.lengths[s] + j, c.cu[b] + j
            pg, at = c.table[s, e // page], e % page
            want["k"][pg, :, at], tol[pg, :, at], want["v"][pg, :, at] = kz[row], bound[row], vn[row]
            want["weights"][pg, :, at], want["stamps"][pg, :, at] = 0, c.counts[s] + j
        if s >= 0:
            lengths[s] += c.cu[b + 1] - c.cu[b]
            counts[s] += c.cu[b + 1] - c.cu[b]
    assert int(c.err.item()) == 0
    got = host(c.k)
    assert np.array_equal(np.isnan(got), np.isnan(want["k"]))
    assert (np.nan_to_num(np.abs(got - want["k"])) <= tol).all()
    for n in ("v", "weights", "stamps"):
        assert np.array_equal(host(getattr(c, n)), want[n], equal_nan=True), n
    assert np.array_equal(c.d_lengths.cpu().numpy(), lengths) and np.array_equal(c.d_counts.cpu().numpy(), counts)
    if with_q:
        z, size = ref.turned(host(c.q), wq if norm else None, 1e-5, 0.0, f, axis, pos, False)
        o, own = host(qo), c.owned()
        for b, s in enumerate(c.slots):
            if s < 0:
                z[c.cu[b]:c.cu[b + 1]] = size[c.cu[b]:c.cu[b + 1]] = 0
        assert (np.abs(o - z) <= ref.turn_bound(z, size, d, dtype))[own].all()
        assert (o[~own] == 7.0).all()
    return c


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("prompts", PROMPTS, ids=str)
def test_append_lengths(dtype, prompts):
    append_case(dtype, prompts)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,rot,page", [(256, 64, 16), (128, 128, 64), (80, 20, 24), (33, 6, 5), (64, 0, 16), (7, 0, 1)])
@pytest.mark.parametrize("kind", ["heads", "places", "joint", "odd"])
def test_append_sizes(dtype, d, rot, page, kind):
    append_case(dtype, [(70, 9), (1, 0), (33, 47)], d=d, rot=rot, page=page, kind=kind, with_q=rot > 0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kw", [dict(axes=3), dict(norm=False), dict(with_q=False), dict(text=True), dict(q_kind="joint"),
                                dict(q_kind="odd"), dict(pad=(1,), gap=6), dict(axes=2, text=True)], ids=str)
def test_append_forms(dtype, kw):
    append_case(dtype, [(70, 9), (20, 3), (33, 47)], **kw)


@pytest.mark.parametrize("B", [300, 1500])
def test_append_of_many_sequences(B):
    r = np.random.default_rng(3)
    append_case("bf16", [(int(r.integers(0, 4)), int(r.integers(0, 20))) for _ in range(B)], Hq=2, Hkv=1, page=8)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what,bit", [("slot", gdn.DEVERR_SLOT), ("room", kv.DEVERR_LENGTH), ("negative", kv.DEVERR_LENGTH),
                                      ("page", kv.DEVERR_PAGE), ("offsets", gdn.DEVERR_SEQLEN)])
def test_append_refusals(dtype, what, bit):
    c = Prompt(41, dtype, [(40, 3), (50, 20), (30, 9)], Hq=4, Hkv=2, d=64, page=16, written=False)
    slot = c.slots[1]
    if what == "slot":
        c.slots[1] = len(c.lengths)
    elif what == "room":
        c.lengths[slot] = c.table.shape[1] * 16 - 49
    elif what == "negative":
        c.lengths[slot] = -3
    elif what == "page":
        c.table[slot, 3] = 10 ** 6
    else:
        c.cu = np.array([0, 40, 30, 120], np.int32)
    c.sync()
    rot = kv.Rotary(frequencies(64))
    qo = torch.full_like(c.q, 7.0)
    before = host(c.k)
    kv.kv_append(c.cache, c.d_slots, c.d_cu, c.kn, c.vn, c.err, rotary=rot, q=c.q, q_out=qo)
    torch.cuda.synchronize()
    assert int(c.err.item()) == bit
    grown = c.d_lengths.cpu().numpy() - c.lengths
    want = np.zeros_like(grown)
    if what != "offsets":
        want[c.slots[0]], want[c.slots[2]] = 40, 30
        assert (qo[:40] != 7.0).any() and (what == "page" or (qo[40:90] == 0).all())
    else:
        assert (qo == 7.0).all() and np.array_equal(host(c.k), before, equal_nan=True)
    assert np.array_equal(grown, want) and np.array_equal(c.d_counts.cpu().numpy() - c.counts, want)
    # nothing but the new entries' places was written
    pages = {int(p) for b in range(3) for p in c.table[c.slots[b] if c.slots[b] < len(c.lengths) else slot]}
    for p in range(before.shape[0]):
        if p not in pages:
            assert np.array_equal(host(c.k[p]), before[p], equal_nan=True)


# ---------------------------------------------------------------- together


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_prompt_in_chunks_then_single_tokens(dtype, d):
    """A prompt appended and attended in two chunks, then two tokens by kv_norm_rotate, kv_tree_attention and
    kv_commit, against the whole text at once."""
    Hq, Hkv, page, n = 8, 2, 16, 230
    dt = TORCH[dtype]
    r = np.random.default_rng(50)
    rows = lambda H: torch.from_numpy(r.normal(size=(n, H, d))).to(dt).cuda()
    q, k, v = rows(Hq), rows(Hkv), rows(Hkv)
    w = torch.from_numpy(1 + 0.1 * r.normal(size=d)).float().cuda()
    rot = kv.Rotary(frequencies(d // 2), q_norm=w, k_norm=w)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")

    def start():
        c = kv.KVCache.allocate(20, Hkv, page, d, 2, 16, dt)
        c.page_table[1, :] = torch.from_numpy(r.permutation(20)[:16].astype(np.int32))
        return c

    def prompt(c, a, b):
        qt, out, lse = torch.empty_like(q[a:b]), torch.empty_like(q[a:b]), torch.empty(b - a, Hq, device="cuda")
        kv.kv_append(c, ints(1), ints(0, b - a), k[a:b], v[a:b], err, rotary=rot, q=q[a:b], q_out=qt)
        kv.kv_prompt_attention(c, ints(1), ints(0, b - a), qt, out, err, kv.kv_prompt_workspace(c, 1, qt), lse=lse)
        return out, lse

    want, wl = prompt(start(), 0, n)
    c = start()
    parts = [prompt(c, 0, 100), prompt(c, 100, 228)]
    for t in (228, 229):
        pos = c.counts[1].view(1, 1).clone()
        qt, kt = torch.empty_like(q[t].view(1, 1, Hq, d)), torch.empty_like(k[t].view(1, 1, Hkv, d))
        kv.kv_norm_rotate(rot, pos, q=q[t].view(1, 1, Hq, d), k=k[t].view(1, 1, Hkv, d), q_out=qt, k_out=kt)
        out, lse = torch.empty_like(qt), torch.empty(1, 1, Hq, device="cuda")
        kv.kv_tree_attention(c, ints(1), qt, kt, v[t].view(1, 1, Hkv, d), kv.tree_masks([[-1]]).cuda(), out, err,
                             kv.kv_tree_workspace(c, qt), lse=lse)
        kv.kv_commit(c, ints(1), kt, v[t].view(1, 1, Hkv, d), ints(0).view(1, 1), ints(1), err)
        parts.append((out[0], lse[0]))
    got, gl = torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])
    assert int(err) == 0 and int(c.lengths[1]) == n == int(c.counts[1])
    # the same keys, queries and values to the bit; the order of sums differs: each side is off by no more than twice
    # the type's rounding of the largest value and 2^-18 of it
    tol = (4 * UNIT[dtype] + 2.0 ** -17) * float(v.abs().max())
    assert (got.float() - want.float()).abs().max().item() <= tol
    assert (gl - wl).abs().max().item() <= 2.0 ** -16 * 8
