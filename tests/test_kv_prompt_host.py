"""Host-only checks of the prompt and page operators' C ABI (include/kv.h): struct layout, refusals before any CUDA
call, the binding's checks. No kernel is launched."""
import ctypes as C
import math
import os
import subprocess
import types

import pytest
import torch

from hybrid_ssm_gated_gb300 import build, gdn, kv
from tests.test_kv_host import ALIGN, BAD_CACHES, DTYPE, FAKE, INCLUDE, NULL, SHAPE, _cache, _rows


@pytest.fixture(scope="module")
def lib():
    build.build()
    return kv.lib()


def _rotary(**over):
    r = kv.kv_rotary(FAKE, FAKE, 0, 0, 1e-6, 0.0, FAKE, FAKE, 32, 1, 0)
    for n, v in over.items():
        setattr(r, n, v)
    return r


def _rotate(lib, rotary=None, dtype=gdn.GDN_BF16, B=2, T=3, Hq=4, Hkv=2, d=64, pos=FAKE, q=True, qo=True, k=True, ko=True):
    row = lambda x: _rows() if x is True else x
    return lib.kv_norm_rotate(rotary or _rotary(), dtype, B, T, Hq, Hkv, d, pos, row(q), row(qo), row(k), row(ko), None)


def _append(lib, c=None, B=2, total=9, Hq=4, slots=FAKE, cu=FAKE, k=True, v=True, rotary=True, pos=FAKE, q=True, qo=True, err=FAKE):
    row = lambda x: _rows() if x is True else x
    return lib.kv_append(c or _cache(), B, total, Hq, slots, cu, row(k), row(v), _rotary() if rotary is True else rotary, pos,
                         row(q), row(qo), err, None)


def _prompt(lib, c=None, B=2, total=9, Hq=4, slots=FAKE, cu=FAKE, q=True, scale=1.0, out=FAKE, lse=FAKE, ws=FAKE, nbytes=0,
            err=FAKE):
    return lib.kv_prompt_attention(c or _cache(), B, total, Hq, slots, cu, _rows() if q is True else q, scale, out, lse, ws,
                                   nbytes, err, None)


def test_struct_layout_matches_the_header(tmp_path):
    fields = [n for n, _ in kv.kv_rotary._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "kv.h"\nint main(void){printf("%zu %d", '
                   'sizeof(kv_rotary), KV_MAX_AXES);'
                   + "".join(f'printf(" %zu", offsetof(kv_rotary, {n}));' for n in fields) + ' return 0;}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", INCLUDE, str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    assert got == [C.sizeof(kv.kv_rotary), kv.MAX_AXES] + [getattr(kv.kv_rotary, n).offset for n in fields]


@pytest.mark.parametrize("over,code", BAD_CACHES, ids=str)
def test_cache_refusals(lib, over, code):
    c = _cache(**over)
    assert _append(lib, c) == code
    assert gdn.gdn_last_error_string().startswith("kv_append")
    assert _prompt(lib, c) == code
    assert lib.kv_fork(c, 2, FAKE, FAKE, FAKE, FAKE, None) == code
    assert lib.kv_compact(c, FAKE, FAKE, 1 << 30, FAKE, None) == code


BAD_ROTARIES = [(dict(rot=3), SHAPE), (dict(rot=-2), SHAPE), (dict(rot=66), SHAPE), (dict(axes=0), SHAPE), (dict(axes=5), SHAPE),
                (dict(turns=None), NULL), (dict(eps=-1.0), SHAPE), (dict(eps=math.nan), SHAPE), (dict(eps=math.inf), SHAPE),
                (dict(offset=math.nan), SHAPE), (dict(q_norm_head=-1), SHAPE), (dict(k_norm_head=-64), SHAPE),
                (dict(q_norm=FAKE + 2), ALIGN), (dict(k_norm=FAKE + 1), ALIGN), (dict(turns=FAKE + 4), ALIGN), (dict(axis=FAKE + 2), ALIGN)]


@pytest.mark.parametrize("over,code", BAD_ROTARIES, ids=str)
def test_rotary_refusals(lib, over, code):
    assert _rotate(lib, _rotary(**over)) == code
    assert _append(lib, rotary=_rotary(**over)) == code


def test_rotate_refusals(lib):
    assert lib.kv_norm_rotate(None, gdn.GDN_BF16, 2, 3, 4, 2, 64, FAKE, _rows(), _rows(), None, None, None) == NULL
    assert _rotate(lib, dtype=3) == DTYPE and _rotate(lib, dtype=-1) == DTYPE
    assert _rotate(lib, d=0) == SHAPE and _rotate(lib, d=257) == SHAPE
    assert _rotate(lib, B=-1) == SHAPE and _rotate(lib, T=-1) == SHAPE and _rotate(lib, B=1 << 20, T=1 << 12) == SHAPE
    assert _rotate(lib, Hq=0) == SHAPE and _rotate(lib, Hkv=0) == SHAPE and _rotate(lib, Hq=(1 << 24) + 1) == SHAPE
    assert _rotate(lib, pos=None) == NULL and _rotate(lib, pos=FAKE + 2) == ALIGN
    assert _rotate(lib, q=None) == NULL and _rotate(lib, ko=None) == NULL
    assert _rotate(lib, q=None, qo=None, k=None, ko=None) == NULL
    for name in ("q", "qo", "k", "ko"):
        assert _rotate(lib, **{name: _rows(p=None)}) == NULL
        assert _rotate(lib, **{name: _rows(head=-1)}) == SHAPE
        assert _rotate(lib, **{name: _rows(p=FAKE + 1)}) == ALIGN
    assert _rotate(lib, B=0) == 0 and _rotate(lib, T=0) == 0


def test_append_refusals(lib):
    assert _append(lib, B=-1) == SHAPE and _append(lib, total=-1) == SHAPE and _append(lib, Hq=0) == SHAPE
    for name in ("slots", "cu", "err"):
        assert _append(lib, **{name: None}) == NULL, name
        assert _append(lib, **{name: FAKE + 2}) == ALIGN, name
    assert _append(lib, pos=FAKE + 1) == ALIGN
    assert _append(lib, qo=None) == NULL and _append(lib, q=None) == NULL and _append(lib, rotary=None) == NULL
    for name in ("q", "qo", "k", "v"):
        assert _append(lib, **{name: _rows(p=None)}) == NULL
        assert _append(lib, **{name: _rows(node=-1)}) == SHAPE
        assert _append(lib, **{name: _rows(p=FAKE + 1)}) == ALIGN
    assert _append(lib, k=None) == NULL and _append(lib, v=None) == NULL
    assert _append(lib, c=_cache(counts=None)) == NULL  # stamps need counts
    assert _append(lib, B=0) == 0


def test_prompt_refusals(lib):
    assert _prompt(lib, B=-1) == SHAPE and _prompt(lib, total=-1) == SHAPE
    assert _prompt(lib, Hq=3) == SHAPE and _prompt(lib, Hq=0) == SHAPE and _prompt(lib, Hq=(1 << 24) + 2) == SHAPE
    assert _prompt(lib, total=1 << 30, Hq=64) == SHAPE  # rows of a key head in 31 bits
    assert _prompt(lib, scale=math.nan) == SHAPE and _prompt(lib, scale=math.inf) == SHAPE
    for name in ("slots", "cu", "out", "ws", "err"):
        assert _prompt(lib, **{name: None}) == NULL, name
    for name, by in (("slots", 2), ("cu", 2), ("out", 1), ("lse", 2), ("ws", 8), ("err", 1)):
        assert _prompt(lib, **{name: FAKE + by}) == ALIGN, name
    assert _prompt(lib, q=_rows(p=None)) == NULL and _prompt(lib, q=_rows(node=-1)) == SHAPE and _prompt(lib, q=None) == NULL
    assert _prompt(lib, B=0) == 0
    assert lib.kv_prompt_attention_workspace(_cache(), 2, -1, 4) == SHAPE
    assert lib.kv_prompt_attention_workspace(_cache(d=300), 2, 3, 4) == SHAPE
    assert lib.kv_prompt_attention_workspace(None, 2, 3, 4) == NULL


def test_page_refusals(lib):
    fork = lambda c=None, n=2, src=FAKE, dst=FAKE, new=FAKE, err=FAKE: lib.kv_fork(c or _cache(), n, src, dst, new, err, None)
    assert fork(n=-1) == SHAPE and fork(n=0) == 0
    for name in ("src", "dst", "new", "err"):
        assert fork(**{name: None}) == NULL and fork(**{name: FAKE + 2}) == ALIGN, name
    comp = lambda c=None, used=FAKE, ws=FAKE, n=1 << 30, err=FAKE: lib.kv_compact(c or _cache(), used, ws, n, err, None)
    assert comp(used=None) == NULL and comp(ws=None) == NULL and comp(err=None) == NULL
    assert comp(used=FAKE + 2) == ALIGN and comp(ws=FAKE + 8) == ALIGN and comp(err=FAKE + 1) == ALIGN
    need = lib.kv_compact_workspace(_cache())
    assert need > 0 and comp(n=need - 1) == SHAPE and "workspace" in gdn.gdn_last_error_string()


def test_turns_of_the_binding():
    """Frequencies as 64-bit fractions of a turn: exact to the last bit of a double, wound to [0, 1) turns."""
    r = kv.Rotary([2 * math.pi / 4, 2 * math.pi * 1.25, 0.0, -2 * math.pi / 4, 1.0], axis=[0, 1, 0, 1, 2], axes=3, device="cpu")
    assert r.turns[:4].tolist() == [1 << 62, 1 << 62, 0, -(1 << 62)] and r.rot == 10
    assert abs(r.turns[4].item() / 2.0 ** 64 - 0.5 / math.pi) < 2.0 ** -54
    assert r.axis.tolist() == [0, 1, 0, 1, 2]


def test_binding_checks_without_a_device():
    for kw in (dict(inv_freq=[math.nan]), dict(inv_freq=[1.0], axis=[0, 0]), dict(inv_freq=[1.0], axis=[1]), dict(axes=0),
               dict(axes=5), dict(q_norm=torch.ones(8)), dict(k_norm=torch.ones(8, dtype=torch.float64))):
        with pytest.raises(ValueError):
            kv.Rotary(device="cpu", **kw)


class Tensor:
    def __init__(self, *shape, dtype=torch.bfloat16, device=1, strides=None):
        self.shape, self.dtype, self.device_index = torch.Size(shape), dtype, device
        self.strides = strides or torch.empty(shape, device="meta").stride()

    def get_device(self):
        return self.device_index

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        return self.strides if i is None else self.strides[i]

    def is_contiguous(self):
        return self.strides == torch.empty(self.shape, device="meta").stride()

    def data_ptr(self):
        return 4096

    def numel(self):
        return self.shape.numel()


def _ints(*shape, device=1):
    return Tensor(*shape, dtype=torch.int32, device=device)


CACHE = types.SimpleNamespace(device=1, dtype=torch.bfloat16, Hkv=2, d=8, _ref=None, page_table=_ints(4, 6))


@pytest.fixture
def calls(monkeypatch):
    """Calls of the library that the binding would make, with the current device at the time."""
    made, now = [], [0]

    class device:
        def __init__(self, i):
            self.i = i

        def __enter__(self):
            self.old, now[0] = now[0], self.i

        def __exit__(self, *x):
            now[0] = self.old

    class Library:
        def __getattr__(self, name):
            return lambda *args: made.append((name, now[0])) or 0

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    monkeypatch.setattr(kv, "lib", lambda: Library())
    return made


def _rot(device=1, axes=1, q_norm=None, k_norm=None):
    r = types.SimpleNamespace(device=device, axes=axes, q_norm=q_norm, k_norm=k_norm, _ref=None)
    r.check = lambda *a: kv.Rotary.check(r, *a)
    return r


def test_calls_go_to_the_caches_device(calls):
    err, ws = _ints(1), Tensor(64, dtype=torch.uint8)
    kv.kv_append(CACHE, _ints(3), _ints(4), Tensor(9, 2, 8), Tensor(9, 2, 8), err, rotary=_rot(), positions=_ints(9),
                 q=Tensor(9, 4, 8), q_out=Tensor(9, 4, 8))
    kv.kv_prompt_attention(CACHE, _ints(3), _ints(4), Tensor(9, 4, 8), Tensor(9, 4, 8), err, ws)
    kv.kv_fork(CACHE, _ints(2), _ints(2), _ints(2, 6), err)
    kv.kv_compact(CACHE, _ints(1), err, ws)
    kv.kv_norm_rotate(_rot(), _ints(2, 3), q=Tensor(2, 3, 4, 8), q_out=Tensor(2, 3, 4, 8))
    assert calls == [(n, 1) for n in ("kv_append", "kv_prompt_attention", "kv_fork", "kv_compact", "kv_norm_rotate")]


@pytest.mark.parametrize("kw", [
    dict(slots=_ints(3, device=0)), dict(cu=_ints(3)), dict(cu=_ints(4, device=0)), dict(k=Tensor(9, 3, 8)), dict(v=Tensor(8, 2, 8)),
    dict(k=Tensor(9, 2, 8, device=0)), dict(v=Tensor(9, 2, 8, dtype=torch.float16)), dict(k=Tensor(9, 2, 8, strides=(32, 16, 2))),
    dict(q=None), dict(q_out=None), dict(rotary=None), dict(rotary=_rot(device=0)), dict(positions=_ints(8)),
    dict(positions=_ints(2, 9)), dict(rotary=_rot(axes=2)), dict(rotary=_rot(k_norm=Tensor(16))),
    dict(rotary=_rot(q_norm=Tensor(2, 8))), dict(q=Tensor(9, 4, 16)), dict(err=_ints(1, device=0))], ids=str)
def test_append_binding_refusals(calls, kw):
    a = dict(slots=_ints(3), cu=_ints(4), k=Tensor(9, 2, 8), v=Tensor(9, 2, 8), err=_ints(1), rotary=_rot(), positions=_ints(9),
             q=Tensor(9, 4, 8), q_out=Tensor(9, 4, 8), **{})
    a.update(kw)
    with pytest.raises(ValueError):
        kv.kv_append(CACHE, a["slots"], a["cu"], a["k"], a["v"], a["err"], rotary=a["rotary"], positions=a["positions"],
                     q=a["q"], q_out=a["q_out"])
    assert not calls


@pytest.mark.parametrize("kw", [
    dict(slots=_ints(3, device=0)), dict(cu=_ints(3)), dict(q=Tensor(9, 4, 16)), dict(q=Tensor(9, 4, 8, device=0)),
    dict(out=Tensor(9, 2, 8)), dict(out=Tensor(9, 4, 8, dtype=torch.float32)), dict(out=Tensor(9, 4, 8, strides=(64, 16, 1))),
    dict(lse=Tensor(9, 4)), dict(lse=Tensor(9, 2, dtype=torch.float32)), dict(ws=Tensor(64, dtype=torch.uint8, device=0))], ids=str)
def test_prompt_binding_refusals(calls, kw):
    a = dict(slots=_ints(3), cu=_ints(4), q=Tensor(9, 4, 8), out=Tensor(9, 4, 8), lse=None, ws=Tensor(64, dtype=torch.uint8))
    a.update(kw)
    with pytest.raises(ValueError):
        kv.kv_prompt_attention(CACHE, a["slots"], a["cu"], a["q"], a["out"], _ints(1), a["ws"], lse=a["lse"])
    assert not calls


def test_other_binding_refusals(calls):
    four = lambda **kw: Tensor(2, 3, 4, 8, **kw)
    bad = [lambda: kv.kv_fork(CACHE, _ints(2), _ints(3), _ints(2, 6), _ints(1)),
           lambda: kv.kv_fork(CACHE, _ints(2), _ints(2), _ints(2, 5), _ints(1)),
           lambda: kv.kv_compact(CACHE, _ints(2), _ints(1), Tensor(64, dtype=torch.uint8)),
           lambda: kv.kv_norm_rotate(_rot(), _ints(2, 3)), lambda: kv.kv_norm_rotate(_rot(), _ints(2, 3), q=four()),
           lambda: kv.kv_norm_rotate(_rot(), _ints(2, 3), q=four(device=0), q_out=four(device=0)),
           lambda: kv.kv_norm_rotate(_rot(), _ints(2, 3), q=four(), q_out=four(dtype=torch.float16)),
           lambda: kv.kv_norm_rotate(_rot(), _ints(2, 3), q=four(dtype=torch.float64), q_out=four(dtype=torch.float64)),
           lambda: kv.kv_norm_rotate(_rot(), _ints(3, 2), q=four(), q_out=four()),
           lambda: kv.kv_norm_rotate(_rot(axes=2), _ints(2, 3), q=four(), q_out=four()),
           lambda: kv.kv_norm_rotate(_rot(q_norm=Tensor(16)), _ints(2, 3), q=four(), q_out=four()),
           lambda: kv.kv_norm_rotate(_rot(), _ints(2, 3), q=four(), q_out=four(), k=Tensor(2, 4, 2, 8), k_out=Tensor(2, 4, 2, 8))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    assert not calls
