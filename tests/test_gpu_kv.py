"""GPU parity of the cache operators of include/kv.h against their definitions in 64 bits
(tests/kv_ref.py): attention of drafted trees, path commit, weight accumulation, eviction.

Every case surrounds the live entries with NaN: entries past a sequence's length, pages nobody holds,
nodes past a sequence's count. Bounds are derived beside the references.
"""
import numpy as np
import pytest
import torch

from hybrid_ssm_gated_gb300 import build, gdn, kv
from tests import kv_ref as ref
from tests.kv_ref import Case, host

pytestmark = pytest.mark.gpu

DTYPES = ["bf16", "f16", "f32"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    kv.lib()


# ---------------------------------------------------------------- attention

# lengths around pages and tiles; every one with several sequences
LENGTHS = [[0, 1, 2], [15, 16, 17, 0], [63, 64, 65, 31], [127, 128, 129, 1], [255, 300, 0, 257]]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens", LENGTHS, ids=str)
@pytest.mark.parametrize("d,page", [(64, 16), (128, 16), (256, 32)])
def test_lengths(dtype, lens, d, page):
    Case(1, dtype, lens, T=3, Hq=4, Hkv=2, d=d, page=page).check_attention()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [1, 2, 7, 8, 16, 33, 64])
@pytest.mark.parametrize("G", [1, 3, 8])
def test_tree_sizes(dtype, T, G):
    Case(2, dtype, [70, 129], T=T, Hq=2 * G, Hkv=2, d=64, page=16, nodes=[T, max(1, T - 1)]).check_attention()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("G", [16, 71, 128, 160])
@pytest.mark.parametrize("d", [64, 256])
def test_many_heads_a_group(dtype, T, G, d):
    """More query heads a key head than a block of rows takes, and numbers that no block divides by."""
    Case(26, dtype, [70, 300], T=T, Hq=G, Hkv=1, d=d, page=16, nodes=[T, max(1, T - 1)]).check_attention()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dims", [(0,), (2,), (0, 1, 2)], ids=str)
def test_rows_shared_by_strides_of_zero(dtype, dims):
    """Drafted keys, values and queries that sequences, heads or all have in common, without a copy."""
    c = Case(27, dtype, [100, 20], T=3, Hq=4, Hkv=2, d=64, page=16)
    for name in ("q", "kn", "vn"):
        x = getattr(c, name)
        for i in dims:
            x = x.narrow(i, 0, 1)
        setattr(c, name, x.expand_as(getattr(c, name)))
    c.check_attention()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [8, 40, 80, 96, 120, 192, 200])
def test_head_sizes(dtype, d):
    Case(3, dtype, [133, 40], T=4, Hq=6, Hkv=3, d=d, page=16).check_attention()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [1, 3, 7, 33, 129, 255])
def test_head_sizes_off_the_grid(dtype, d):
    Case(4, dtype, [66, 5], T=3, Hq=4, Hkv=2, d=d, page=8).check_attention()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("page", [1, 5, 8, 24, 48, 64, 100, 128, 256])
def test_page_sizes(dtype, page):
    Case(5, dtype, [300, 131, 7], T=2, Hq=4, Hkv=2, d=64, page=page).check_attention()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["heads", "places", "joint", "odd"])
def test_cache_layouts(dtype, kind):
    Case(6, dtype, [150, 33], T=5, Hq=4, Hkv=2, d=64, page=16, kind=kind).check_attention()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shift", [0, 1])
def test_rows_of_one_projection(dtype, shift):
    """q, k and v as parts of one wider row (shift 1: off the 16-byte grid)."""
    c = Case(7, dtype, [100, 20], T=4, Hq=4, Hkv=2, d=64, page=16)
    wide = torch.full((2, 4, (4 + 2 + 2) * 64 + 16), float("nan"), dtype=c.q.dtype, device="cuda")
    parts = [wide[..., shift:][..., a * 64:(a + n) * 64].unflatten(-1, (n, 64)) for a, n in ((0, 4), (4, 2), (6, 2))]
    for p, x in zip(parts, (c.q, c.kn, c.vn)):
        p.copy_(x)
    plain, _ = c.attend()
    c.q, c.kn, c.vn = parts
    out, _ = c.check_attention()
    if shift == 0:
        assert torch.equal(out, plain)


@pytest.mark.parametrize("dtype", DTYPES)
def test_nodes_of_each_sequence(dtype):
    c = Case(8, dtype, [20, 0, 140, 9, 0], T=9, Hq=4, Hkv=2, d=64, page=16, nodes=[9, 3, 0, 1, 0], pad=(3,))
    out, lse = c.check_attention()
    for b, n in ((0, 9), (1, 3), (2, 0), (3, 0), (4, 0)):
        assert (out[b, n:] == 0).all() and (lse[b, n:] == float("-inf")).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_masks_of_every_kind(dtype):
    """Rows that attend nothing of the tree, later nodes, everything, and bits past the count."""
    c = Case(9, dtype, [0, 40], T=6, Hq=4, Hkv=2, d=64, page=16, nodes=[4, 6])
    c.mask[:] = np.array([[0, 0b1000, 0b1111, (1 << 64) - 1, 1, 1], [0, 1 << 5, (1 << 64) - 1, 1 << 63, 0b11, 0]],
                         np.uint64)
    c.sync()
    out, lse = c.check_attention()
    assert (out[0, 0] == 0).all() and (lse[0, 0] == float("-inf")).all()  # no cache, empty mask


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_values_that_a_row_does_not_attend(dtype, value):
    """A node with NaN or infinite key and value reaches the rows that attend it and no others."""
    c = Case(10, dtype, [30, 0], T=4, Hq=4, Hkv=2, d=64, page=16)
    c.mask[:] = np.array([0b0001, 0b0011, 0b0101, 0b1001], np.uint64)
    c.vn[:, 2] = value
    c.kn[:, 3] = float("nan")
    c.sync()
    out, lse = c.attend()
    o, want = host(out), c.reference()[0]
    assert int(c.err.item()) == 0
    assert np.isfinite(o[:, :2]).all()
    _, _, mag, smag = c.reference()
    assert (np.abs(o[:, :2] - want[:, :2]) <= ref.out_bound(mag, smag, 64, dtype)[:, :2]).all()
    assert (np.isnan(o[:, 2]).all() if np.isnan(value) else np.isinf(o[:, 2]).all())
    assert np.isnan(o[:, 3]).all() and np.isnan(host(lse)[:, 3]).all()
    assert np.isfinite(host(lse)[:, :3]).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_large_scores(dtype):
    """Scores of hundreds, whose maximum moves from tile to tile, both ways."""
    c = Case(11, dtype, [700, 333], T=3, Hq=4, Hkv=2, d=64, page=16, spread=6.0)
    c.check_attention()
    c.scale = -c.scale
    c.check_attention()
    c.scale = 0.0
    c.check_attention()


@pytest.mark.parametrize("dtype", DTYPES)
def test_scores_that_grow(dtype):
    """Each tile's scores lie far above the last one's, then far below."""
    c = Case(12, dtype, [1000, 900], T=2, Hq=4, Hkv=2, d=64, page=16)
    for b, up in ((0, 1), (1, -1)):
        for e in range(c.lengths[c.slots[b]]):
            pg = int(c.table[c.slots[b], e // 16])
            c.k[pg, :, e % 16, 0] = up * (e // 64) * 8.0
    c.q[..., 0] = 8.0
    c.sync()
    c.check_attention()


@pytest.mark.parametrize("dtype", DTYPES)
def test_many_sequences(dtype):
    """More sequences than the kernels' blocks have threads, some of them padding."""
    r = np.random.default_rng(3)
    lens = [int(x) for x in r.integers(0, 12, 700)]
    Case(13, dtype, lens, T=1, Hq=2, Hkv=1, d=32, page=8, pad=tuple(range(5, 700, 9))).check_attention()


@pytest.mark.parametrize("dtype", DTYPES)
def test_long_sequences_over_many_blocks(dtype):
    c = Case(14, dtype, [5000, 1, 2600], T=5, Hq=8, Hkv=2, d=64, page=64)
    a, za = c.check_attention()
    b, zb = c.attend()
    assert torch.equal(a, b) and torch.equal(za, zb)  # one order of additions


@pytest.mark.parametrize("dtype", DTYPES)
def test_one_unit_over_the_whole_grid(dtype):
    """A single key head of one long sequence: more partial results than a warp has lanes."""
    Case(19, dtype, [21003], T=2, Hq=2, Hkv=1, d=64, page=64).check_attention()


@pytest.mark.parametrize("dtype", DTYPES)
def test_scores_beyond_the_rounding_of_one(dtype):
    """Scores near 1e9, whose own rounding is dozens: the largest still takes the row."""
    c = Case(24, dtype, [300], T=2, Hq=2, Hkv=1, d=64, page=16)
    c.q[:], c.kn[:] = 0, 0
    c.q[..., 0] = 30000.0
    c.k[torch.from_numpy(c.table[c.slots[0], :19]).long()] = 0
    for e in range(300):  # entry 271 leads by far
        c.k[int(c.table[c.slots[0], e // 16]), :, e % 16, 0] = 30000.0 if e == 271 else 20000.0 - e
    c.scale = 1.0
    c.sync()
    out, lse = c.attend()
    want = host(c.v[int(c.table[c.slots[0], 271 // 16]), 0, 271 % 16])
    assert (np.abs(host(out) - want) <= 2 * ref.UNIT[dtype] * np.abs(want) + 1e-6).all()
    assert np.isfinite(host(lse)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_calls_in_a_graph(dtype):
    """Every call can be captured (none synchronises or allocates) and replayed on new contents."""
    c = Case(25, dtype, [60, 200], T=3, Hq=4, Hkv=2, d=64, page=16, room=3)
    plain, lse = c.attend()
    out, lse = torch.empty_like(plain), torch.empty_like(lse)
    ws, ev = kv.kv_tree_workspace(c.cache, c.q), kv.kv_evict_workspace(c.cache, 2, 100)
    path = torch.tensor([[0, 1], [0, 2]], dtype=torch.int32, device="cuda")
    n = torch.tensor([2, 1], dtype=torch.int32, device="cuda")
    want = c.pools()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        kv.kv_tree_attention(c.cache, c.d_slots, c.q, c.kn, c.vn, c.d_mask, out, c.err, ws, lse=lse, scale=c.scale)
        kv.kv_commit(c.cache, c.d_slots, c.kn, c.vn, path, n, c.err)
        kv.kv_accumulate(c.cache, c.d_slots, c.q, lse, path, n, c.err, scale=c.scale)
        kv.kv_evict(c.cache, c.d_slots, 100, 20, c.err, ev)
    c.assert_pools(want)  # capturing ran nothing
    graph.replay()
    torch.cuda.synchronize()
    assert int(c.err.item()) == 0 and torch.equal(out, plain)
    assert c.d_lengths[c.d_slots.long()].tolist() == [62, 100]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_optional_outputs_and_counts(dtype):
    c = Case(15, dtype, [90, 4], T=3, Hq=4, Hkv=2, d=64, page=16)
    a, _ = c.attend()
    b, none = c.attend(with_nodes=False, with_lse=False)
    assert none is None and torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_another_stream(dtype):
    c = Case(16, dtype, [400, 70], T=3, Hq=4, Hkv=2, d=64, page=16)
    a, _ = c.attend()
    s = torch.cuda.Stream()
    b, _ = c.attend(stream=s)
    with torch.cuda.stream(s):
        d, _ = c.attend()
    assert torch.equal(a, b) and torch.equal(a, d)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_refused_sequences(dtype):
    """A slot, a length, a page or a node count out of range: error bits, zero outputs, the others right."""
    c = Case(17, dtype, [50, 60, 70, 80, 90], T=3, Hq=4, Hkv=2, d=64, page=16)
    good = c.attend()[0]
    c.table[c.slots[1], 2] = c.k.shape[0]
    c.lengths[c.slots[2]] = c.table.shape[1] * 16 + 1
    c.nodes[3] = 4
    c.slots[4] = c.table.shape[0]
    c.sync()
    out, lse = c.attend()
    assert int(c.err.item()) == gdn.DEVERR_SLOT | kv.DEVERR_LENGTH | kv.DEVERR_PAGE | kv.DEVERR_NODES
    assert torch.equal(out[0], good[0])
    assert (out[1:] == 0).all() and (lse[1:] == float("-inf")).all()
    c.err.zero_()
    c.table[c.slots[1], 2] = -1
    c.lengths[c.slots[2]], c.nodes[3] = -1, -1
    c.sync()
    out, _ = c.attend()
    assert int(c.err.item()) == gdn.DEVERR_SLOT | kv.DEVERR_LENGTH | kv.DEVERR_PAGE | kv.DEVERR_NODES
    assert torch.equal(out[0], good[0]) and (out[1:] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16"])
def test_offsets_past_32_bits(dtype):
    """Pages more than 2^32 bytes, and 2^31 elements, into the pool."""
    page, H, d = 64, 2, 128
    num = (1 << 31) // (page * H * d) + 8
    k = torch.empty(num, H, page, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    c = Case(18, dtype, [page * 3 + 5], T=2, Hq=4, Hkv=H, d=d, page=page, room=8)
    want, _ = c.attend()
    used = c.table[c.slots[0], :4].copy()
    for i, far in enumerate((num - 1, 0, num - 3, num - 2)):
        k[far], v[far] = c.k[int(used[i])], c.v[int(used[i])]
        c.table[c.slots[0], i] = far
    c.k, c.v = k, v
    c.weights = torch.zeros(num, H, page, device="cuda")
    c.stamps = torch.zeros(num, H, page, dtype=torch.int32, device="cuda")
    c.sync()
    got, _ = c.attend()
    assert torch.equal(got, want)
    path = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    kv.kv_commit(c.cache, c.d_slots, c.kn, c.vn, path, torch.tensor([2], dtype=torch.int32, device="cuda"), c.err)
    assert int(c.err.item()) == 0
    assert torch.equal(k[num - 2, :, 5:7], c.kn[0].transpose(0, 1)) and int(c.d_lengths[c.slots[0]]) == page * 3 + 7


# ---------------------------------------------------------------- commit


def _paths(c, P, npath):
    path = np.stack([c.r.permutation(max(P, c.T))[:P] % c.T for _ in range(c.B)]).astype(np.int32)
    return path, np.array(npath, np.int32)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind,d,page", [("heads", 64, 16), ("places", 128, 8), ("joint", 40, 5), ("odd", 33, 16)])
def test_commit(dtype, kind, d, page):
    c = Case(20, dtype, [0, 15, 16, 40, 7], T=6, Hq=2, Hkv=2, d=d, page=page, kind=kind, room=6, pad=(3,))
    path, npath = _paths(c, 5, [5, 3, 1, 4, 0])
    want = c.pools()
    lengths, counts = c.lengths.copy(), c.counts.copy()
    ref.commit(want, c.table, lengths, counts, c.slots, host(c.kn), host(c.vn), path, npath)
    dev = lambda a: torch.from_numpy(a).cuda()
    kv.kv_commit(c.cache, c.d_slots, c.kn, c.vn, dev(path), dev(npath), c.err)
    assert int(c.err.item()) == 0
    c.assert_pools(want)
    assert np.array_equal(c.d_lengths.cpu().numpy(), lengths) and np.array_equal(c.d_counts.cpu().numpy(), counts)


def test_commit_refusals():
    """No room, a missing page, a path out of range: nothing of that sequence is written."""
    c = Case(21, "bf16", [10, 30, 5, 6, 7], T=4, Hq=2, Hkv=2, d=64, page=16, room=4)
    path = np.tile(np.arange(4, dtype=np.int32), (5, 1))
    npath = np.array([2, 4, 2, 5, 2], np.int32)
    c.table[c.slots[1], 2] = -1  # entries 30, 31 fit; 32, 33 do not
    path[2, 1] = 4
    c.slots[4] = c.table.shape[0] + 3
    c.sync()
    want = c.pools()
    lengths, counts = c.lengths.copy(), c.counts.copy()
    ref.commit(want, c.table, lengths, counts, c.slots[:1], host(c.kn), host(c.vn), path, npath)
    dev = lambda a: torch.from_numpy(a).cuda()
    kv.kv_commit(c.cache, c.d_slots, c.kn, c.vn, dev(path), dev(npath), c.err)
    assert int(c.err.item()) == kv.DEVERR_PAGE | kv.DEVERR_NODES | gdn.DEVERR_SLOT
    c.assert_pools(want)
    assert np.array_equal(c.d_lengths.cpu().numpy(), lengths)
    c.err.zero_()
    c.lengths[c.slots[0]] = c.table.shape[1] * 16 - 1  # one entry of room
    c.sync()
    kv.kv_commit(c.cache, c.d_slots[:1], c.kn[:1], c.vn[:1], dev(path[:1]), dev(npath[:1]), c.err)
    assert int(c.err.item()) == kv.DEVERR_LENGTH


# ---------------------------------------------------------------- accumulation


def _accumulate(c, path, npath, decay, lse):
    before = c.weights.cpu().numpy().astype(np.float64)
    want, tol = ref.accumulate(host(c.k), before, c.table, c.lengths, c.slots, host(c.q), host(lse), path, npath,
                               c.scale, decay)
    dev = lambda a: torch.from_numpy(a).cuda()
    kv.kv_accumulate(c.cache, c.d_slots, c.q, lse, dev(path), dev(npath), c.err, decay=decay, scale=c.scale)
    got = c.weights.cpu().numpy().astype(np.float64)
    off = np.abs(got - want)
    assert (off <= tol).all(), f"weights off by {off.max():.3e}"
    assert np.array_equal(got[tol == 0], before[tol == 0])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,page,kind", [(64, 16, "heads"), (128, 48, "places"), (80, 16, "joint"), (256, 64, "heads"),
                                         (33, 7, "odd")])
@pytest.mark.parametrize("G", [1, 4])
def test_accumulate(dtype, d, page, kind, G):
    lens = [3, 64, 129, 300, 40, 65]
    c = Case(30, dtype, lens, T=6, Hq=2 * G, Hkv=2, d=d, page=page, kind=kind, pad=(4,))
    path, npath = _paths(c, 3, [3, 1, 2, 3, 2, 0])
    lse = torch.from_numpy(c.r.normal(size=(6, 6, 2 * G)) + 4).float().cuda()
    lse[1, path[1, 0], 0] = float("-inf")
    _accumulate(c, path, npath, 0.75, lse)
    assert int(c.err.item()) == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("G", [16, 71, 160])
@pytest.mark.parametrize("d", [64, 256])
def test_accumulate_many_heads_a_group(dtype, G, d):
    c = Case(35, dtype, [200, 41], T=3, Hq=G, Hkv=1, d=d, page=16)
    path, npath = _paths(c, 2, [2, 1])
    _accumulate(c, path, npath, 1.0, torch.full((2, 3, G), 5.0, device="cuda"))


@pytest.mark.parametrize("dtype", DTYPES)
def test_accumulate_long_paths(dtype):
    """Paths of up to 40 nodes of a group of 8 heads: more rows than one block takes."""
    c = Case(31, dtype, [200, 41], T=64, Hq=8, Hkv=1, d=64, page=16)
    path, npath = _paths(c, 40, [40, 17])
    _accumulate(c, path, npath, 1.0, torch.full((2, 64, 8), 5.0, device="cuda"))


@pytest.mark.parametrize("dtype", DTYPES)
def test_commit_then_accumulate_is_the_attention_given(dtype):
    """After a commit of a root-to-leaf path the weights of each head sum to rows x group size, and the
    log-sum-exps of the tree step are those of the committed sequence."""
    c = Case(32, dtype, [0, 37, 200], T=5, Hq=4, Hkv=2, d=64, page=16, room=5)
    c.mask[:] = np.array([0b1, 0b11, 0b101, 0b1011, 0b11011], np.uint64)
    c.sync()
    _, lse = c.attend()
    path = np.tile(np.array([0, 1, 3, 4], np.int32), (3, 1))
    npath = np.array([4, 3, 4], np.int32)
    dev = lambda a: torch.from_numpy(a).cuda()
    kv.kv_commit(c.cache, c.d_slots, c.kn, c.vn, dev(path), dev(npath), c.err)
    c.weights.zero_()
    kv.kv_accumulate(c.cache, c.d_slots, c.q, lse, dev(path), dev(npath), c.err, scale=c.scale)
    assert int(c.err.item()) == 0
    w = c.weights.double().cpu().numpy()
    for b in range(3):
        L = c.lengths[c.slots[b]] + npath[b]
        total = ref.entries(w[..., None], c.table, c.slots[b], 0, L).sum()
        assert abs(total - 2 * npath[b]) < 1e-4 * 2 * npath[b]


@pytest.mark.parametrize("dtype", DTYPES)
def test_accumulate_many_sequences(dtype):
    r = np.random.default_rng(5)
    lens = [int(x) for x in r.integers(2, 12, 700)]
    c = Case(34, dtype, lens, T=2, Hq=2, Hkv=1, d=32, page=8, pad=tuple(range(3, 700, 10)))
    path, npath = _paths(c, 2, [int(x) for x in r.integers(0, 3, 700)])
    _accumulate(c, path, npath, 0.5, torch.full((700, 2, 2), 2.0, device="cuda"))
    assert int(c.err.item()) == 0


def test_accumulate_refusals():
    c = Case(33, "bf16", [20, 2, 30, 40], T=4, Hq=2, Hkv=2, d=64, page=16)
    path = np.tile(np.arange(4, dtype=np.int32), (4, 1))
    npath = np.array([2, 3, 2, 2], np.int32)  # the second sequence holds two entries only
    path[2, 1] = -1
    c.table[c.slots[3], 1] = 1 << 20
    c.sync()
    before = c.weights.clone()
    dev = lambda a: torch.from_numpy(a).cuda()
    lse = torch.zeros(4, 4, 2, device="cuda")
    kv.kv_accumulate(c.cache, c.d_slots, c.q, lse, dev(path), dev(npath), c.err, scale=c.scale)
    assert int(c.err.item()) == kv.DEVERR_LENGTH | kv.DEVERR_NODES | kv.DEVERR_PAGE
    mine = c.table[c.slots[0], :2]
    rest = np.setdiff1d(np.arange(c.k.shape[0]), mine)
    assert torch.equal(c.weights[rest], before[rest]) and not torch.equal(c.weights[mine], before[mine])


# ---------------------------------------------------------------- eviction


def _evict(c, budget, recent):
    want = c.pools()
    lengths = c.lengths.copy()
    ref.evict(want, c.table, lengths, c.counts, c.slots, budget, recent)
    ws = kv.kv_evict_workspace(c.cache, c.B, budget)
    ws.view(torch.int32).fill_(-12345)
    kv.kv_evict(c.cache, c.d_slots, budget, recent, c.err, ws)
    assert int(c.err.item()) == 0
    c.assert_pools(want)
    assert np.array_equal(c.d_lengths.cpu().numpy(), lengths)


def _scramble(c, ages=True):
    """Stamps of each head a random order of the newest counts (as after earlier evictions)."""
    for b, slot in enumerate(c.slots):
        if slot < 0:
            continue
        L = int(c.lengths[slot])
        for h in range(c.Hkv):
            order = c.r.permutation(L) + int(c.counts[slot]) - L
            for e in range(L):
                c.stamps[int(c.table[slot, e // c.page]), h, e % c.page] = int(order[e])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (64, 10), (100, 100), (255, 0), (300, 17), (2000, 5)])
def test_evict(dtype, budget, recent):
    c = Case(40, dtype, [0, 1, 100, 256, 301, 64], T=1, Hq=2, Hkv=2, d=64, page=16, pad=(3,))
    _scramble(c)
    _evict(c, budget, recent)


@pytest.mark.parametrize("kind,d,page", [("places", 128, 8), ("joint", 40, 5), ("odd", 33, 16), ("heads", 256, 48)])
def test_evict_layouts(kind, d, page):
    c = Case(41, "bf16", [90, 201, 30], T=1, Hq=2, Hkv=2, d=d, page=page, kind=kind)
    _scramble(c)
    _evict(c, 77, 20)


@pytest.mark.parametrize("weights", ["equal", "few", "signs", "special", "tiny"])
def test_evict_ties_and_special_weights(weights):
    """Ties go to the lowest entry; NaN counts as the largest weight; -0 ties with 0."""
    c = Case(42, "f16", [400, 130], T=1, Hq=2, Hkv=2, d=32, page=16)
    w = torch.ones_like(c.weights)
    r = torch.from_numpy(c.r.integers(0, 6, size=tuple(w.shape))).cuda()
    if weights == "few":
        w = r.float()
    elif weights == "signs":
        w = torch.tensor([0.0, -0.0, 1.0, -1.0, -2.0, 2.0], device="cuda")[r]
    elif weights == "special":
        w = torch.tensor([float("nan"), float("inf"), float("-inf"), 3e38, 0.0, -float("nan")], device="cuda")[r]
    elif weights == "tiny":
        w = r.float() * 1e-45
    c.weights.copy_(w)
    _scramble(c)
    _evict(c, 100, 30)


def test_evict_long():
    """One long sequence, and the moves spread over many blocks."""
    c = Case(43, "bf16", [9000], T=1, Hq=1, Hkv=1, d=8, page=16)
    _scramble(c)
    _evict(c, 4000, 100)


def test_evict_refusals():
    c = Case(44, "bf16", [60, 70, 80], T=1, Hq=2, Hkv=2, d=64, page=16)
    _scramble(c)
    c.table[c.slots[0], 1] = c.k.shape[0]
    c.lengths[c.slots[1]] = 1 << 20
    c.slots[2] = 99
    c.sync()
    want = c.pools()
    ws = kv.kv_evict_workspace(c.cache, 3, 50)
    kv.kv_evict(c.cache, c.d_slots, 50, 5, c.err, ws)
    assert int(c.err.item()) == kv.DEVERR_PAGE | kv.DEVERR_LENGTH | gdn.DEVERR_SLOT
    c.assert_pools(want)
    assert np.array_equal(c.d_lengths.cpu().numpy(), c.lengths)


def test_evict_offsets_past_32_bits():
    """Pages more than 2^31 elements into the pools of keys and values."""
    page, H, d = 64, 2, 128
    num = (1 << 31) // (page * H * d) + 6
    c = Case(45, "bf16", [page * 3], T=1, Hq=2, Hkv=H, d=d, page=page)
    _scramble(c)
    want = c.pools()
    lengths = c.lengths.copy()
    ref.evict(want, c.table, lengths, c.counts, c.slots, 100, 10)
    used, far = c.table[c.slots[0], :3].copy(), [num - 2, 1, num - 1]
    k = torch.empty(num, H, page, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    w = torch.zeros(num, H, page, device="cuda")
    s = torch.zeros(num, H, page, dtype=torch.int32, device="cuda")
    for i, f in enumerate(far):
        u = int(used[i])
        k[f], v[f], w[f], s[f] = c.k[u], c.v[u], c.weights[u], c.stamps[u]
        c.table[c.slots[0], i] = f
    c.k, c.v, c.weights, c.stamps = k, v, w, s
    c.sync()
    kv.kv_evict(c.cache, c.d_slots, 100, 10, c.err, kv.kv_evict_workspace(c.cache, 1, 100))
    assert int(c.err.item()) == 0
    for i, f in enumerate(far):
        u = int(used[i])
        assert np.array_equal(host(k[f]), want["k"][u]) and np.array_equal(host(v[f]), want["v"][u])
        assert np.array_equal(w[f].cpu().numpy(), want["weights"][u]) and np.array_equal(s[f].cpu().numpy(), want["stamps"][u])


# ---------------------------------------------------------------- together


def test_speculative_decoding_gives_the_tokens_of_plain_decoding():
    """The example: verified trees of a hybrid model against one token at a time, and with a budget."""
    from examples import hybrid_tree_verify as ex

    plain, said, rounds, tree = ex.run(batch=3, steps=40)
    assert int(tree.err.item()) == 0 and plain == said and rounds < 40
    _, _, _, tree = ex.run(batch=2, steps=60, budget=32, recent=8)
    assert int(tree.err.item()) == 0
    assert tree.cache.lengths.tolist() == [32, 32] and min(tree.cache.counts.tolist()) >= 60
