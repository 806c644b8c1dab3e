"""GPU parity of the page operators of include/kv.h with a simulation on the host: forks of sequences and the
compaction of the pool. Everything is compared bit for bit, what must not change too."""
import numpy as np
import pytest
import torch

from hybrid_ssm_gated_gb300 import build, gdn, kv
from tests.kv_ref import TORCH, host, layout

pytestmark = pytest.mark.gpu

DTYPES = ["bf16", "f16", "f32"]
NAMES = ("k", "v", "weights", "stamps")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    kv.lib()


class Pool:
    """A cache of sequences of the given lengths (0: an ended one) in random pages, with spare slots and pages."""

    def __init__(self, seed, dtype, lens, Hkv, d, page, kind="heads", spare=8, extra_slots=6, books=True):
        r = self.r = np.random.default_rng(seed)
        need = [-(-n // page) for n in lens]
        slots, pages, self.max_pages = len(lens) + extra_slots, sum(need) + spare, max(need + [1]) + 2
        self.page, self.dtype = page, dtype
        self.slots = r.permutation(slots).astype(np.int32)
        order, at = r.permutation(pages), 0
        self.table = r.integers(-9, 3 * pages, size=(slots, self.max_pages)).astype(np.int32)  # past a length: anything
        self.lengths = np.zeros(slots, np.int32)
        for b, n in enumerate(lens):
            self.table[self.slots[b], :need[b]] = order[at:at + need[b]]
            at += need[b]
            self.lengths[self.slots[b]] = n
        self.free = list(order[at:])
        self.counts = self.lengths + 5
        self.k, self.v = layout((pages, Hkv, page, d), dtype, kind)
        for x in (self.k, self.v):
            x.copy_(torch.from_numpy(r.normal(size=(pages, Hkv, page, d))).to(TORCH[dtype]))
        shape = (pages, Hkv, page)
        self.weights = torch.from_numpy(r.exponential(size=shape)).float().cuda() if books else None
        self.stamps = torch.from_numpy(r.integers(0, 99, size=shape)).int().cuda() if books else None
        self.books, self.err = books, torch.zeros(1, dtype=torch.int32, device="cuda")
        self.sync()

    def sync(self):
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
        self.d_table, self.d_lengths, self.d_counts = dev(self.table), dev(self.lengths), dev(self.counts)
        self.cache = kv.KVCache(self.k, self.v, self.d_table, self.d_lengths, self.d_counts, self.weights, self.stamps)

    def pools(self):
        return {n: host(getattr(self, n)).copy() for n in (NAMES if self.books else NAMES[:2])}

    def assert_is(self, pools):
        for n, x in pools.items():
            assert np.array_equal(host(getattr(self, n)), x), n
        assert np.array_equal(self.d_table.cpu().numpy(), self.table)
        assert np.array_equal(self.d_lengths.cpu().numpy(), self.lengths)
        assert np.array_equal(self.d_counts.cpu().numpy(), self.counts)


def fork(p, src, dst, new, refused=()):
    """The fork on the host (into p's tables and the returned pools) and on the device, compared."""
    pools = p.pools()
    d_new = torch.from_numpy(new).cuda()
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    kv.kv_fork(p.cache, ints(src), ints(dst), d_new, p.err)
    torch.cuda.synchronize()
    for i, (s, t) in enumerate(zip(src, dst)):
        if s < 0 or t < 0 or i in refused:
            continue
        n = int(p.lengths[s])
        for j in range(-(-n // p.page)):
            old, fresh = p.table[s, j], new[i, j]
            if fresh >= 0:
                live = min(p.page, n - j * p.page)
                for x in pools.values():
                    x[fresh, :, :live] = x[old, :, :live]
            p.table[t, j] = fresh if fresh >= 0 else old
        p.lengths[t], p.counts[t] = n, p.counts[s]
    p.assert_is(pools)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens", [[1], [16, 17, 15], [100, 0, 48], [700, 33]], ids=str)
@pytest.mark.parametrize("whole", [False, True])
def test_fork(dtype, lens, whole):
    need = sum(-(-n // 16) for n in lens)
    p = Pool(60, dtype, lens, Hkv=2, d=64, page=16, spare=2 * need + 4, extra_slots=2 * len(lens) + 1)
    src = [int(p.slots[i % len(lens)]) for i in range(2 * len(lens))]
    dst = [int(x) for x in p.slots[len(lens):3 * len(lens)]]
    new = np.full((len(src), p.max_pages), -1, np.int32)
    for i, s in enumerate(src):
        n = int(p.lengths[s])
        for j in range(n // 16 if not whole and n % 16 else 0 if whole else -(-n // 16), -(-n // 16)):
            new[i, j] = p.free.pop()
    fork(p, src, dst, new)
    assert int(p.err.item()) == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,page,kind", [(64, 16, "places"), (64, 16, "joint"), (33, 5, "heads"), (64, 24, "odd"), (256, 64, "heads"),
                                         (255, 1, "heads"), (1, 128, "heads")])
@pytest.mark.parametrize("books", [True, False])
def test_fork_layouts(dtype, d, page, kind, books):
    p = Pool(61, dtype, [90, 31], Hkv=3, d=d, page=page, kind=kind, spare=200, books=books)
    new = np.where(np.random.default_rng(1).random((2, p.max_pages)) < 0.5, -1, 0).astype(np.int32)
    for i in range(2):
        for j in range(p.max_pages):
            if new[i, j] == 0:
                new[i, j] = p.free.pop()
    fork(p, [int(p.slots[0]), int(p.slots[1])], [int(p.slots[2]), int(p.slots[3])], new)
    assert int(p.err.item()) == 0


@pytest.mark.parametrize("what,bit", [("src", gdn.DEVERR_SLOT), ("dst", gdn.DEVERR_SLOT), ("itself", gdn.DEVERR_SLOT),
                                      ("length", kv.DEVERR_LENGTH), ("negative", kv.DEVERR_LENGTH), ("page", kv.DEVERR_PAGE),
                                      ("new page", kv.DEVERR_PAGE), ("padding", 0)])
def test_fork_refusals(what, bit):
    """One of three forks is refused, or none of its slots is one; the others are made."""
    p = Pool(62, "bf16", [70, 40, 50], Hkv=2, d=64, page=16, spare=12)
    src, dst = [int(x) for x in p.slots[:3]], [int(x) for x in p.slots[3:6]]
    new = np.full((3, p.max_pages), -1, np.int32)
    for i in range(3):
        new[i, (int(p.lengths[src[i]]) - 1) // 16] = p.free.pop()
    if what == "src":
        src[1] = len(p.lengths)
    elif what == "dst":
        dst[1] = len(p.lengths)
    elif what == "itself":
        dst[1] = src[1]
    elif what == "length":
        p.lengths[src[1]] = p.max_pages * 16 + 1
    elif what == "negative":
        p.lengths[src[1]] = -1
    elif what == "page":
        p.table[src[1], 0] = p.k.shape[0]
    elif what == "new page":
        new[1, 1] = p.k.shape[0]
    else:
        src[1] = -1
    p.sync()
    fork(p, src, dst, new, refused=(1,))
    assert int(p.err.item()) == bit


def compact(p):
    """The compaction on the host and on the device, compared; pages held."""
    pools = p.pools()
    used = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    ws = kv.kv_compact_workspace(p.cache).fill_(0xA5)
    kv.kv_compact(p.cache, used, p.err, ws)
    torch.cuda.synchronize()
    held = {int(x) for s, n in enumerate(p.lengths) for x in p.table[s, :-(-int(n) // p.page)]}
    U = len(held)
    holes, movers = sorted(set(range(U)) - held), sorted(x for x in held if x >= U)
    to = dict(zip(movers, holes))
    for a, b in to.items():
        for x in pools.values():
            x[b] = x[a]
    for s, n in enumerate(p.lengths):
        for j in range(-(-int(n) // p.page)):
            p.table[s, j] = to.get(int(p.table[s, j]), p.table[s, j])
    p.assert_is(pools)
    assert int(used.item()) == U and int(p.err.item()) == 0
    return U, len(holes)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens", [[1], [0, 0], [100, 0, 48, 7], [16 * 40, 0, 33, 0, 16 * 20]], ids=str)
@pytest.mark.parametrize("spare", [0, 1, 31, 90])
def test_compact(dtype, lens, spare):
    p = Pool(63, dtype, lens, Hkv=2, d=64, page=16, spare=spare + (0 if sum(lens) else 1))
    compact(p)
    assert compact(p)[1] == 0  # the second time nothing moves


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,page,kind", [(64, 16, "places"), (64, 16, "joint"), (33, 5, "heads"), (64, 24, "odd"), (256, 64, "heads"),
                                         (255, 1, "heads")])
@pytest.mark.parametrize("books", [True, False])
def test_compact_layouts(dtype, d, page, kind, books):
    assert compact(Pool(64, dtype, [90, 31, 0, 60], Hkv=3, d=d, page=page, kind=kind, spare=100, books=books))[1] > 0


@pytest.mark.parametrize("pages", [31, 32, 33, 1023, 1024, 1025, 40000])
def test_compact_of_many_pages(pages):
    """Counts of pages around the words and threads of the plan; more slots than warps."""
    r = np.random.default_rng(pages)
    lens, left = [], pages * 2 // 3
    while left > 0:
        n = min(left, int(r.integers(1, 40)))
        lens.append(4 * n - int(r.integers(0, 4)))
        left -= n
    p = Pool(65, "bf16", lens, Hkv=1, d=8, page=4, spare=pages - sum(-(-n // 4) for n in lens))
    drop = r.random(len(p.lengths)) < 0.4
    p.lengths[drop] = 0
    p.sync()
    compact(p)


def test_compact_of_shared_pages():
    """A page that several sequences hold moves once, and all of them follow."""
    p = Pool(66, "bf16", [70, 40, 50], Hkv=2, d=64, page=16, spare=30)
    src, dst = [int(x) for x in p.slots[:3]], [int(x) for x in p.slots[3:6]]
    fork(p, src, dst, np.full((3, p.max_pages), -1, np.int32))
    p.lengths[src[1]] = 0
    p.sync()
    compact(p)


@pytest.mark.parametrize("what,bit", [("length", kv.DEVERR_LENGTH), ("negative", kv.DEVERR_LENGTH), ("page", kv.DEVERR_PAGE),
                                      ("below", kv.DEVERR_PAGE)])
def test_compact_refusals(what, bit):
    p = Pool(67, "bf16", [70, 40, 50], Hkv=2, d=64, page=16, spare=30)
    if what == "length":
        p.lengths[p.slots[1]] = p.max_pages * 16 + 1
    elif what == "negative":
        p.lengths[p.slots[4]] = -1
    else:
        p.table[p.slots[1], 1] = p.k.shape[0] if what == "page" else -1
    p.sync()
    pools = p.pools()
    used = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv.kv_compact(p.cache, used, p.err, kv.kv_compact_workspace(p.cache))
    torch.cuda.synchronize()
    assert int(used.item()) == -1 and int(p.err.item()) == bit
    p.assert_is(pools)


def test_captured_compaction_behind_a_fork():
    """A graph of both, replayed over changed tables."""
    p = Pool(68, "bf16", [70, 40, 50], Hkv=2, d=64, page=16, spare=30)
    src, dst = [int(p.slots[0])], [int(p.slots[3])]
    new = np.full((1, p.max_pages), -1, np.int32)
    new[0, 4] = p.free.pop()
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    a, b, d_new, used = ints(src), ints(dst), torch.from_numpy(new).cuda(), ints([0])
    ws = kv.kv_compact_workspace(p.cache)
    start = {n: getattr(p, n).clone() for n in NAMES + ("d_table", "d_lengths", "d_counts")}
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()

    def call():
        kv.kv_fork(p.cache, a, b, d_new, p.err)
        kv.kv_compact(p.cache, used, p.err, ws)

    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    want = {n: getattr(p, n).clone() for n in start}
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        for n, x in start.items():
            getattr(p, n).copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(getattr(p, n), x) for n, x in want.items()) and int(used) == 13 and int(p.err) == 0


@pytest.mark.parametrize("extra_slots,spare", [(6, 50), (4000, 50), (6, (1 << 18) + 5)])
def test_compact_forms(extra_slots, spare):
    """Tables and pools that one block marks, and those that a grid marks: many slots, many pages."""
    lens = [0 if i % 3 == 2 else 3 + 7 * i for i in range(40)]
    p = Pool(69, "bf16", lens, Hkv=1, d=8, page=4, spare=spare, extra_slots=extra_slots)
    assert compact(p)[1] > 0
    p.lengths[p.slots[5]] = -4
    p.sync()
    used = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv.kv_compact(p.cache, used, p.err, kv.kv_compact_workspace(p.cache))
    assert int(used.item()) == -1 and int(p.err.item()) == kv.DEVERR_LENGTH
