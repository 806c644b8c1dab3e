"""Prompts and page operators in a pool whose offsets pass 32 bits in elements and bytes, everything compared to the bit."""
import pytest
import torch

from hybrid_ssm_gated_gb300 import build, kv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    kv.lib()


@pytest.mark.parametrize("page,d", [(64, 128), (24, 100)], ids=["16-byte pieces", "2-byte pieces"])
def test_append_fork_and_compaction_past_4_gib(page, d):
    Hkv, n = 2, 250
    num = (1 << 32) // (Hkv * page * d) + 40
    held = -(-n // page)
    k, v = (torch.zeros(num, Hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    weights, stamps = torch.zeros(num, Hkv, page, device="cuda"), torch.zeros(num, Hkv, page, dtype=torch.int32, device="cuda")
    assert (num - 20) * k.stride(0) > 1 << 32
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    table = torch.full((3, held + 2), -1, dtype=torch.int32, device="cuda")
    far = [num - 1 - j for j in range(held)]
    table[1, :held] = i32(*far)
    c = kv.KVCache(k, v, table, i32(0, 0, 0), i32(0, 9, 0), weights, stamps)
    g = torch.Generator(device="cuda").manual_seed(page)
    kn, vn = (torch.randn(n, Hkv, d, device="cuda", generator=g).bfloat16() for _ in range(2))
    err = i32(0)

    def rows(pool, slot):
        x = pool[c.page_table[slot, :held].long()]  # [pages, Hkv, page, ...]
        return x.transpose(1, 2).reshape(held * page, Hkv, *x.shape[3:])[:n]

    def check(slot):
        assert torch.equal(rows(k, slot), kn) and torch.equal(rows(v, slot), vn)
        assert torch.equal(rows(stamps, slot), (9 + torch.arange(n, device="cuda")).int()[:, None].expand(n, Hkv))
        assert torch.equal(rows(weights, slot), want_weights)

    # two appends
    want_weights = torch.zeros(n, Hkv, device="cuda")
    weights.fill_(3.0)
    for a, b in ((0, 100), (100, n)):
        kv.kv_append(c, i32(1), i32(0, b - a), kn[a:b], vn[a:b], err)
    assert c.lengths.tolist() == [0, n, 0] and int(err) == 0
    check(1)
    for j in range(held):  # a weight of its own for every entry
        weights[far[j]] = torch.rand(Hkv, page, device="cuda", generator=g)
    want_weights = rows(weights, 1).clone()
    # a fork with pages of its own, then one that shares all but the last
    new = torch.full((1, held + 2), -1, dtype=torch.int32, device="cuda")
    new[0, :held] = i32(*[num - 20 - 2 * j for j in range(held)])
    kv.kv_fork(c, i32(1), i32(2), new, err)
    new.fill_(-1)
    new[0, held - 1] = num - 15
    kv.kv_fork(c, i32(1), i32(0), new, err)
    assert c.lengths.tolist() == [n] * 3 and c.counts.tolist() == [9 + n] * 3 and int(err) == 0
    for slot in range(3):
        check(slot)
    assert c.page_table[0, :held].tolist() == far[:-1] + [num - 15]
    # the pool's front: contents of the pages, whole, where the tables then say
    names = (k, v, weights, stamps)
    old = c.page_table[:, :held].clone()
    before = [x[old.flatten().long()].clone() for x in names]
    used = i32(0)
    kv.kv_compact(c, used, err, kv.kv_compact_workspace(c))
    U = 2 * held + 1
    assert int(used) == U and int(err) == 0 and sorted(set(c.page_table[:, :held].flatten().tolist())) == list(range(U))
    now = c.page_table[:, :held].flatten().long()
    assert all(torch.equal(x[now], b) for x, b in zip(names, before))
    to = {a: i for i, a in enumerate(sorted(set(old.flatten().tolist())))}  # movers in order take holes in order
    assert [to[x] for x in old.flatten().tolist()] == now.tolist()
    for slot in range(3):
        check(slot)
