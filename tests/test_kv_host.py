"""Host-only checks of the cache's C ABI (include/kv.h): struct layout, exports, refusals before any CUDA
call, the binding's checks. No kernel is launched."""
import ctypes as C
import os
import re
import subprocess

import pytest
import torch

from hybrid_ssm_gated_gb300 import build, gdn, kv

FAKE = 0x7F0000000000  # 16-byte aligned stand-in pointer; never dereferenced on these paths
INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return kv.lib()


def test_every_declared_function_is_exported(lib):
    text = open(os.path.join(INCLUDE, "kv.h")).read()
    names = set(re.findall(r"^(?:int|int64_t)\s+(kv_[a-z_]+)\(", text, re.M))
    assert names == set(kv._SIGS)
    for n in names:
        assert hasattr(lib, n)


def test_struct_layout_and_constants_match_the_header(tmp_path):
    fields = [n for n, _ in kv.kv_cache._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "kv.h"\nint main(void){printf("%zu %zu", '
                   'sizeof(kv_cache), sizeof(kv_rows));'
                   + "".join(f'printf(" %zu", offsetof(kv_cache, {n}));' for n in fields)
                   + "".join(f'printf(" %zu", offsetof(kv_rows, {n}));' for n, _ in kv.kv_rows._fields_)
                   + 'printf(" %d %d %d %d %d", KV_DEVERR_LENGTH, KV_DEVERR_PAGE, KV_DEVERR_NODES, KV_MAX_NODES, '
                   'KV_MAX_D); return 0;}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", INCLUDE, str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    want = [C.sizeof(kv.kv_cache), C.sizeof(kv.kv_rows)] + [getattr(kv.kv_cache, n).offset for n in fields] + \
        [getattr(kv.kv_rows, n).offset for n, _ in kv.kv_rows._fields_] + \
        [kv.DEVERR_LENGTH, kv.DEVERR_PAGE, kv.DEVERR_NODES, kv.MAX_NODES, kv.MAX_D]
    assert got == want


def _cache(**over):
    c = kv.kv_cache(FAKE, FAKE, gdn.GDN_BF16, 2, 16, 64, 8, 2048, 1024, 64, 2048, 1024, 64, FAKE, 4, 4, FAKE, FAKE, FAKE,
                    FAKE)
    for n, v in over.items():
        setattr(c, n, v)
    return c


def _rows(**over):
    r = kv.kv_rows(FAKE, 512, 256, 64)
    for n, v in over.items():
        setattr(r, n, v)
    return r


def _attend(lib, c=None, B=2, T=3, Hq=4, slots=FAKE, q=None, kn=None, vn=None, mask=FAKE, nodes=FAKE, scale=1.0, out=FAKE,
            lse=FAKE, ws=FAKE, nbytes=0, err=FAKE):
    return lib.kv_tree_attention(c or _cache(), B, T, Hq, slots, q or _rows(), kn or _rows(), vn or _rows(), mask, nodes,
                                 scale, out, lse, ws, nbytes, err, None)


NULL, DTYPE, SHAPE, WINDOW, ALIGN = -1, -2, -3, -4, -5
BAD_CACHES = [(dict(k=None), NULL), (dict(v=None), NULL), (dict(page_table=None), NULL), (dict(lengths=None), NULL),
              (dict(dtype=3), DTYPE), (dict(Hkv=0), SHAPE), (dict(page_size=0), SHAPE), (dict(d=0), SHAPE),
              (dict(d=257), SHAPE), (dict(num_pages=-1), SHAPE), (dict(max_pages=1 << 28), SHAPE),
              (dict(num_slots=-1), SHAPE), (dict(k_token=-64), SHAPE), (dict(v_head=-1), SHAPE), (dict(k=FAKE + 1), ALIGN),
              (dict(lengths=FAKE + 2), ALIGN), (dict(weights=None), NULL)]


@pytest.mark.parametrize("over,code", BAD_CACHES, ids=str)
def test_cache_refusals(lib, over, code):
    c = _cache(**over)
    assert _attend(lib, c) == code
    assert gdn.gdn_last_error_string().startswith("kv_tree_attention")
    assert lib.kv_commit(c, 2, 3, 2, FAKE, _rows(), _rows(), FAKE, FAKE, FAKE, None) == code
    assert lib.kv_accumulate(c, 2, 3, 2, 4, FAKE, _rows(), FAKE, FAKE, FAKE, 1.0, 1.0, FAKE, None) == code
    assert lib.kv_evict(c, 2, FAKE, 4, 1, FAKE, 1 << 30, FAKE, None) == code


def test_attention_refusals(lib):
    assert lib.kv_tree_attention(None, 2, 3, 4, FAKE, _rows(), _rows(), _rows(), FAKE, FAKE, 1.0, FAKE, FAKE, FAKE, 0, FAKE,
                                 None) == NULL
    assert _attend(lib, T=0) == WINDOW and _attend(lib, T=65) == WINDOW
    assert _attend(lib, Hq=3) == SHAPE and _attend(lib, Hq=0) == SHAPE and _attend(lib, B=-1) == SHAPE
    assert _attend(lib, Hq=(1 << 24) + 2) == SHAPE
    assert _attend(lib, scale=float("nan")) == SHAPE and _attend(lib, scale=float("inf")) == SHAPE
    for name in ("slots", "mask", "out", "ws", "err"):
        assert _attend(lib, **{name: None}) == NULL, name
    for name in ("q", "kn", "vn"):
        assert _attend(lib, **{name: _rows(p=None)}) == NULL
        assert _attend(lib, **{name: _rows(node=-1)}) == SHAPE
        assert _attend(lib, **{name: _rows(p=FAKE + 1)}) == ALIGN
    for name, by in (("slots", 2), ("mask", 4), ("nodes", 2), ("out", 1), ("lse", 2), ("ws", 8), ("err", 1)):
        assert _attend(lib, **{name: FAKE + by}) == ALIGN, name
    assert _attend(lib, B=0) == 0
    assert lib.kv_tree_attention_workspace(_cache(), 2, 65, 4) == WINDOW
    assert lib.kv_tree_attention_workspace(_cache(d=300), 2, 3, 4) == SHAPE


def test_commit_and_accumulate_refusals(lib):
    commit = lambda c=None, B=2, T=3, P=2, slots=FAKE, kn=None, vn=None, path=FAKE, n=FAKE, err=FAKE: lib.kv_commit(
        c or _cache(), B, T, P, slots, kn or _rows(), vn or _rows(), path, n, err, None)
    assert commit(T=0) == WINDOW and commit(P=0) == WINDOW and commit(P=65) == WINDOW
    assert commit(slots=None) == NULL and commit(path=None) == NULL and commit(n=None) == NULL and commit(err=None) == NULL
    assert commit(kn=_rows(p=None)) == NULL and commit(vn=_rows(p=FAKE + 1)) == ALIGN
    assert commit(c=_cache(counts=None)) == NULL  # stamps need counts
    assert commit(path=FAKE + 2) == ALIGN and commit(B=0) == 0
    acc = lambda c=None, B=2, T=3, P=2, Hq=4, q=None, lse=FAKE, path=FAKE, n=FAKE, scale=1.0, decay=1.0: lib.kv_accumulate(
        c or _cache(), B, T, P, Hq, FAKE, q or _rows(), lse, path, n, scale, decay, FAKE, None)
    assert acc(Hq=5) == SHAPE and acc(P=0) == WINDOW and acc(decay=float("nan")) == SHAPE
    assert acc(lse=None) == NULL and acc(lse=FAKE + 2) == ALIGN and acc(B=0) == 0
    assert acc(c=_cache(weights=None, stamps=None)) == NULL


def test_evict_refusals(lib):
    ev = lambda c=None, B=2, slots=FAKE, budget=40, recent=4, ws=FAKE, n=1 << 20, err=FAKE: lib.kv_evict(
        c or _cache(), B, slots, budget, recent, ws, n, err, None)
    assert ev(budget=0) == SHAPE and ev(recent=-1) == SHAPE and ev(recent=41) == SHAPE and ev(B=-1) == SHAPE
    assert ev(slots=None) == NULL and ev(ws=None) == NULL and ev(c=_cache(counts=None)) == NULL
    assert ev(ws=FAKE + 8) == ALIGN
    need = lib.kv_evict_workspace(_cache(), 2, 40)
    assert need > 0 and ev(n=need - 1) == SHAPE and "workspace" in gdn.gdn_last_error_string()
    assert ev(budget=64, recent=0, n=1 << 20) == 0  # the table holds 64 entries at most: nothing to do
    assert ev(B=0) == 0


def test_tree_masks():
    m = kv.tree_masks([[-1, 0, 0, 2], [-1, -1, 1, 0]])
    assert m.tolist() == [[1, 3, 5, 13], [1, 2, 6, 9]]
    chain = kv.tree_masks([list(range(-1, 63))])
    assert chain[0, 63].item() == -1 and chain[0, 62].item() == (1 << 63) - 1
    with pytest.raises(ValueError):
        kv.tree_masks([[0]])


def test_binding_checks_without_a_device():
    k = torch.zeros(2, 1, 4, 8)
    with pytest.raises(ValueError):  # not a CUDA tensor
        kv.KVCache(k, k, torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        kv.KVCache(k, k.double(), torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
