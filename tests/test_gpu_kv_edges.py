"""GPU parity of the cache operators of include/kv.h where their inputs or sizes are extreme: long sums, weights
far below a leader's, paths of more than 2^31 pieces, infinite keys, rows without a log-sum-exp. References in
64 bits, as tests/test_gpu_kv.py.
"""
import numpy as np
import pytest
import torch

from hybrid_ssm_gated_gb300 import build, kv
from tests import kv_ref as ref
from tests.kv_ref import Case, host

pytestmark = pytest.mark.gpu

DTYPES = ["bf16", "f16", "f32"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    kv.lib()


dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ---------------------------------------------------------------- attention


def _one_text(dtype, T, gap, n=131072, page=128, d=64):
    """Attention over n entries of which the first leads the others, all alike, by `gap`: outputs, log-sum-exps
    and what both should be. Enough sequences (of one text, so that the pool is two pages) that a block of the
    device takes a whole one."""
    B = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    dt = ref.TORCH[dtype]
    k, v = torch.zeros(2, 1, page, d, dtype=dt, device="cuda"), torch.zeros(2, 1, page, d, dtype=dt, device="cuda")
    k[0, 0, 0, 0] = gap
    gap = float(k[0, 0, 0, 0])  # as the cache holds it
    tail = torch.linspace(0.5, 2.0, d, device="cuda").to(dt)
    v[:] = tail
    v[0, 0, 0] = 1.0
    table = torch.ones(1, n // page, dtype=torch.int32, device="cuda")
    table[0, 0] = 0
    cache = kv.KVCache(k, v, table, torch.full((1,), n, dtype=torch.int32, device="cuda"))
    q = torch.zeros(B, T, 1, d, dtype=dt, device="cuda")
    q[..., 0] = 1.0
    new = torch.zeros(B, T, 1, d, dtype=dt, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(B, T, 1, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv.kv_tree_attention(cache, torch.zeros(B, dtype=torch.int32, device="cuda"), q, new, new,
                         torch.zeros(B, T, dtype=torch.int64, device="cuda"), out, err, kv.kv_tree_workspace(cache, q),
                         lse=lse, scale=1.0)
    assert int(err.item()) == 0
    rest = (n - 1) * np.exp(-gap)
    return host(out), host(lse), (1.0 + rest * host(tail)) / (1.0 + rest), gap + np.log1p(rest), gap


def _check_one_text(dtype, out, lse, want, z, gap, n=131072, d=64):
    """Beside the bound of any row, the sums': of 2048 entries at most in tensor memory, which cuts off at 2^-24
    at worst; on the FP32 pipe of 64, and of the tiles."""
    mag, smag = np.broadcast_to(want, out.shape), np.full(lse.shape, gap)
    sums = (64 + n / 64) * 2.0 ** -24 if dtype == "f32" else 2048 * 2.0 ** -24
    off = np.abs(out - want)
    assert (off <= ref.out_bound(mag, smag, d, dtype) + sums * mag).all(), f"outputs off by {off.max():.3e}"
    assert (np.abs(lse - z) <= ref.lse_bound(np.full(lse.shape, z), smag, d)).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("gap", [0.0, 2.0, 4.0, 8.0])
def test_sums_over_long_caches(dtype, T, gap):
    """Outputs do not shrink with the number of like entries that are summed."""
    _check_one_text(dtype, *_one_text(dtype, T, gap))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("gap", [12.0, 14.0, 16.0, 16.96875, 17.46875, 18.0])
def test_many_entries_far_below_one(dtype, T, gap):
    """One entry leads 131071 others, each of which weighs 2^-17 to 2^-26 of it: too little for fp16 beside a
    weight of one, and together up to half of the row."""
    _check_one_text(dtype, *_one_text(dtype, T, gap))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("T,G", [(1, 1), (5, 5), (50, 2)])
@pytest.mark.parametrize("moves", [0, 1])
def test_whole_sequences_of_many_tiles(dtype, d, T, G, moves):
    """A block of the device takes a sequence whole, 43 tiles of 128 entries, for every size of a block of rows
    and of a head; moves: the maximum rises again and again on the way."""
    n, page, B = 5500, 128, 2 * torch.cuda.get_device_properties(0).multi_processor_count
    dt, g = ref.TORCH[dtype], torch.Generator(device="cuda").manual_seed(60)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    pages = -(-n // page)
    k, v = rnd(pages, 1, page, d), rnd(pages, 1, page, d)
    if moves:
        k *= 1.0 + 3.0 * (torch.arange(pages, device="cuda") // 5 / (pages // 5)).view(-1, 1, 1, 1)
    k, v = k.to(dt), v.to(dt)
    order = torch.randperm(pages, generator=g, device="cuda").int().view(1, pages)
    cache = kv.KVCache(k, v, order, torch.full((1,), n, dtype=torch.int32, device="cuda"))
    q, kn, vn = rnd(1, T, G, d).to(dt), rnd(1, T, 1, d).to(dt), rnd(1, T, 1, d).to(dt)
    mask = torch.ones(1, T, dtype=torch.int64, device="cuda").expand(B, T).contiguous()  # every node sees the first
    out, lse = torch.empty(B, T, G, d, dtype=dt, device="cuda"), torch.empty(B, T, G, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    many = lambda x: x.expand(B, -1, -1, -1).contiguous()
    kv.kv_tree_attention(cache, torch.zeros(B, dtype=torch.int32, device="cuda"), many(q), many(kn), many(vn), mask, out,
                         err, kv.kv_tree_workspace(cache, out), lse=lse)
    assert int(err.item()) == 0
    at = order[0].long()
    keys = torch.cat([k[at, 0].reshape(-1, d)[:n], kn[0, :1, 0]]).double()
    vals = torch.cat([v[at, 0].reshape(-1, d)[:n], vn[0, :1, 0]]).double()
    s = q[0].double() @ keys.T / d ** 0.5
    p = s.softmax(-1)
    want, mag, z = host(p @ vals), host(p @ vals.abs()), host(s.logsumexp(-1))
    smag = host((q[0].double().abs() @ keys.abs().T).amax(-1) / d ** 0.5)
    assert (np.abs(host(out) - want) <= ref.out_bound(mag, smag, d, dtype)).all()
    assert (np.abs(host(lse) - z) <= ref.lse_bound(z, smag, d)).all()


# ---------------------------------------------------------------- commit


@pytest.mark.parametrize("n", [1, 64])
def test_commit_of_more_pieces_than_32_bits(n):
    """32768 key heads of fp32 rows off the 16-byte grid: 2^31 pieces of two bytes, or a call that could have them."""
    H, T, d = 32768, 64, 256
    k, v = (torch.full((1, H, T, d + 1), float("nan"), device="cuda")[..., 1:] for _ in range(2))
    zeros = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    w = torch.full((1, H, T), 5.0, device="cuda")
    cache = kv.KVCache(k, v, zeros(1, 1), zeros(1), zeros(1) + 7, w, zeros(1, H, T))
    g = torch.Generator(device="cuda").manual_seed(80)
    kn, vn = (torch.randn(1, T, 1, d, generator=g, device="cuda").expand(1, T, H, d) for _ in range(2))
    path = torch.randperm(T, generator=g, device="cuda").int().view(1, T)
    err = zeros(1)
    kv.kv_commit(cache, zeros(1), kn, vn, path, zeros(1) + n, err)
    assert int(err.item()) == 0 and cache.lengths.tolist() == [n] and cache.counts.tolist() == [7 + n]
    at = path[0, :n].long()
    for pool, new in ((k, kn), (v, vn)):
        assert (pool[0, :, :n] == new[0, at, 0]).all() and pool[0, :, n:].isnan().all()
    assert (w[0, :, :n] == 0).all() and (w[0, :, n:] == 5).all()
    assert (cache.stamps[0, :, :n] == torch.arange(7, 7 + n, device="cuda")).all()


# ---------------------------------------------------------------- accumulation


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("G,P", [(1, 1), (4, 3), (5, 5), (8, 12)])
@pytest.mark.parametrize("d", [64, 192])
def test_accumulate_infinite_keys(dtype, G, P, d):
    """An entry whose scores are all -inf gathers nothing and one of +inf everything, however many rows the
    path has beside a kernel's block of them; the other entries do not notice."""
    c = Case(50, dtype, [140, 33], T=P, Hq=2 * G, Hkv=2, d=d, page=16)
    path = np.stack([c.r.permutation(P) for _ in range(2)]).astype(np.int32)
    npath = np.array([P, 1], np.int32)
    c.q[..., 0] = c.q[..., 0].abs() + 1.0  # the sign of an infinite score is that of the key's first element
    at = lambda b, e: (int(c.table[c.slots[b], e // 16]), slice(None), e % 16)
    low, high = [(0, 0), (0, 77), (1, 5)], [(0, 20), (1, 31)]
    k, before = host(c.k), c.weights.cpu().numpy().astype(np.float64)  # the reference sees finite keys
    want, tol = ref.accumulate(k, before, c.table, c.lengths, c.slots, host(c.q), np.full((2, P, 2 * G), 3.0), path, npath,
                               c.scale, 0.5)
    for (entries, value) in ((low, float("-inf")), (high, float("inf"))):
        for b, e in entries:
            c.k[at(b, e) + (0,)] = value
            want[at(b, e)] = before[at(b, e)] * 0.5 if value < 0 else np.inf
            tol[at(b, e)] = 0
    lse = torch.full((2, P, 2 * G), 3.0, device="cuda")
    kv.kv_accumulate(c.cache, c.d_slots, c.q, lse, dev(path), dev(npath), c.err, decay=0.5, scale=c.scale)
    got = c.weights.cpu().numpy().astype(np.float64)
    assert int(c.err.item()) == 0
    fin = np.isfinite(want)
    assert np.array_equal(got[~fin], want[~fin])
    assert (np.abs(got[fin] - want[fin]) <= tol[fin]).all(), f"weights off by {np.abs(got[fin] - want[fin]).max():.3e}"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
def test_accumulate_rows_without_a_log_sum_exp(dtype, poison):
    """A row whose log-sum-exp is -inf adds nothing, whatever its query and the keys hold."""
    c = Case(51, dtype, [200, 20], T=3, Hq=4, Hkv=2, d=64, page=16)
    path, npath = np.tile(np.arange(3, dtype=np.int32), (2, 1)), np.array([3, 2], np.int32)
    lse = torch.full((2, 3, 4), 4.0, device="cuda")
    lse[0, 1], lse[1, 0, 2] = float("-inf"), float("-inf")
    before = c.weights.cpu().numpy().astype(np.float64)
    want, tol = ref.accumulate(host(c.k), before, c.table, c.lengths, c.slots, host(c.q), host(lse), path, npath, c.scale, 1.0)
    c.q[0, 1], c.q[1, 0, 2] = poison, poison
    kv.kv_accumulate(c.cache, c.d_slots, c.q, lse, dev(path), dev(npath), c.err, scale=c.scale)
    got = c.weights.cpu().numpy().astype(np.float64)
    assert int(c.err.item()) == 0
    assert (np.abs(got - want) <= tol).all()


# ---------------------------------------------------------------- eviction


@pytest.mark.parametrize("weights", ["random", "few"])
@pytest.mark.parametrize("H,lens,page", [(3, [20001], 16),            # clusters of eight
                                         (50, [9003, 4200], 16),      # of two (a hundred units)
                                         (25, [9003, 8800], 20),      # of four
                                         (40, [9003, 70], 6),         # of two, entries one by one
                                         (80, [50001, 300], 16),      # one block a unit, more keys than it holds
                                         (80, [46081, 46080], 5),     # and entries one by one
                                         (2, [400003], 16)],          # clusters of eight, more than their blocks hold
                         ids=str)
def test_evict_in_slices_of_every_kind(H, lens, page, weights):
    """The selection by one block to eight a unit, with its keys in shared memory and formed again and again, to
    the bit; few: ties over all slices, the threshold among them."""
    r = np.random.default_rng(90)
    d, B, need = 2, len(lens), [-(-n // page) for n in lens]
    num = sum(need) + 1
    order = r.permutation(num).astype(np.int32)
    table = np.full((B, max(need) + 1), -5, np.int32)
    table[0, :need[0]] = order[:need[0]]
    if B > 1:
        table[1, :need[1]] = order[need[0]:sum(need)]
    k, v = (r.normal(size=(num, H, page, d)).astype(np.float16) for _ in range(2))
    w = r.exponential(size=(num, H, page)) if weights == "random" else r.integers(0, 3, size=(num, H, page))
    w = w.astype(np.float32)
    s = r.integers(0, max(lens), size=(num, H, page)).astype(np.int32)
    counts = np.array(lens, np.int32) + 3
    budget, recent = max(lens) * 2 // 5, max(lens) // 50
    dk, dv, dw, ds = dev(k), dev(v), dev(w), dev(s)
    cache = kv.KVCache(dk, dv, dev(table), dev(np.array(lens, np.int32)), dev(counts), dw, ds)
    for b, L in enumerate(lens):
        if L <= budget:
            continue
        e = np.arange(L)
        pg, at = table[b, e // page], e % page
        for h in range(H):
            x, st = w[pg, h, at], s[pg, h, at]
            best = np.lexsort((e, -x, st < counts[b] - recent))[:budget]  # kept by age first, then weight, then place
            kept = np.zeros(L, bool)
            kept[best] = True
            holes, fill = np.flatnonzero(~kept[:budget]), budget + np.flatnonzero(kept[budget:])
            # (among those kept by age the lowest entry goes first, whatever its weight; they are fewer than the budget)
            assert len(holes) == len(fill) > 0 and (st >= counts[b] - recent).sum() < budget
            for a in (k, v, w, s):
                a[pg[holes], h, at[holes]] = a[pg[fill], h, at[fill]]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = kv.kv_evict_workspace(cache, B, budget)
    ws.view(torch.int32).fill_(-12345)
    kv.kv_evict(cache, torch.arange(B, dtype=torch.int32, device="cuda"), budget, recent, err, ws)
    assert int(err.item()) == 0 and cache.lengths.tolist() == [min(n, budget) for n in lens]
    for got, want in ((dk, k), (dv, v), (dw, w), (ds, s)):
        assert np.array_equal(got.cpu().numpy(), want)
