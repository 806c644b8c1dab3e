"""Thin ctypes binding of the key/value cache's C ABI in include/kv.h.

Like the binding of gdn.h (hybrid_ssm_gated_gb300/gdn.py): functions carry the
C entry points' names and only marshal arguments; every step runs in libgdn.so,
and there is no fallback.
"""
from __future__ import annotations

import ctypes as C
import math

import torch

from . import gdn
from .gdn import DTYPE_CODE, _check, _ptr
from .gdn import _stream as _given_stream

DEVERR_LENGTH, DEVERR_PAGE, DEVERR_NODES = 64, 128, 256
MAX_NODES, MAX_D, MAX_AXES = 64, 256, 4


class kv_cache(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("dtype", C.c_int32), ("Hkv", C.c_int32),
                ("page_size", C.c_int32), ("d", C.c_int32), ("num_pages", C.c_int64), ("k_page", C.c_int64),
                ("k_head", C.c_int64), ("k_token", C.c_int64), ("v_page", C.c_int64), ("v_head", C.c_int64),
                ("v_token", C.c_int64), ("page_table", C.c_void_p), ("max_pages", C.c_int32),
                ("num_slots", C.c_int64), ("lengths", C.c_void_p), ("counts", C.c_void_p), ("weights", C.c_void_p),
                ("stamps", C.c_void_p)]


class kv_rows(C.Structure):
    _fields_ = [("p", C.c_void_p), ("seq", C.c_int64), ("node", C.c_int64), ("head", C.c_int64)]


class kv_rotary(C.Structure):
    _fields_ = [("q_norm", C.c_void_p), ("k_norm", C.c_void_p), ("q_norm_head", C.c_int64), ("k_norm_head", C.c_int64),
                ("eps", C.c_float), ("offset", C.c_float), ("turns", C.c_void_p), ("axis", C.c_void_p),
                ("rot", C.c_int32), ("axes", C.c_int32), ("interleaved", C.c_int32)]


_P, _I, _F, _L = C.c_void_p, C.c_int32, C.c_float, C.c_int64
_CACHE, _ROWS, _ROTARY = C.POINTER(kv_cache), C.POINTER(kv_rows), C.POINTER(kv_rotary)
_SIGS = {
    "kv_tree_attention": ([_CACHE, _I, _I, _I, _P, _ROWS, _ROWS, _ROWS, _P, _P, _F, _P, _P, _P, _L, _P, _P], C.c_int),
    "kv_tree_attention_workspace": ([_CACHE, _I, _I, _I], _L),
    "kv_commit": ([_CACHE, _I, _I, _I, _P, _ROWS, _ROWS, _P, _P, _P, _P], C.c_int),
    "kv_accumulate": ([_CACHE, _I, _I, _I, _I, _P, _ROWS, _P, _P, _P, _F, _F, _P, _P], C.c_int),
    "kv_evict": ([_CACHE, _I, _P, _I, _I, _P, _L, _P, _P], C.c_int),
    "kv_evict_workspace": ([_CACHE, _I, _I], _L),
    "kv_norm_rotate": ([_ROTARY, _I, _I, _I, _I, _I, _I, _P, _ROWS, _ROWS, _ROWS, _ROWS, _P], C.c_int),
    "kv_append": ([_CACHE, _I, _I, _I, _P, _P, _ROWS, _ROWS, _ROTARY, _P, _ROWS, _ROWS, _P, _P], C.c_int),
    "kv_prompt_attention": ([_CACHE, _I, _I, _I, _P, _P, _ROWS, _F, _P, _P, _P, _L, _P, _P], C.c_int),
    "kv_prompt_attention_workspace": ([_CACHE, _I, _I, _I], _L),
    "kv_fork": ([_CACHE, _I, _P, _P, _P, _P, _P], C.c_int),
    "kv_compact": ([_CACHE, _P, _P, _L, _P, _P], C.c_int),
    "kv_compact_workspace": ([_CACHE], _L),
}
_lib = None


def lib() -> C.CDLL:
    """The loaded libgdn.so (gdn.lib()) with the signatures of include/kv.h."""
    global _lib
    if _lib is None:
        lib_ = gdn.lib()
        for name, (args, res) in _SIGS.items():
            fn = getattr(lib_, name)
            fn.argtypes, fn.restype = args, res
        _lib = lib_
    return _lib


def _pages(t: torch.Tensor, name: str):
    if not t.is_cuda or t.dim() != 4 or t.stride(3) != 1:
        raise ValueError(f"kv: {name} must be a CUDA tensor [num_pages, Hkv, page_size, d] with unit stride in d")
    return t.stride(0), t.stride(1), t.stride(2)


class KVCache:
    """Device tensors of one attention layer's cache (layouts as in include/kv.h).

    k, v [num_pages, Hkv, page_size, d], any strides with d contiguous (a [num_pages, page_size, Hkv, d]
    pool is passed as its transpose(1, 2)); page_table [num_slots, max_pages], lengths and counts
    [num_slots] int32; weights fp32 and stamps int32 [num_pages, Hkv, page_size], or None where
    nothing is accumulated or evicted.
    """

    def __init__(self, k, v, page_table, lengths, counts=None, weights=None, stamps=None):
        if k.shape != v.shape or k.dtype != v.dtype or k.dtype not in DTYPE_CODE:
            raise ValueError("kv: k and v must have one shape and one of the dtypes float32, bfloat16, float16")
        k_strides, v_strides = _pages(k, "k"), _pages(v, "v")
        num_pages, Hkv, page_size, d = k.shape
        if page_table.dim() != 2 or lengths.shape != page_table.shape[:1]:
            raise ValueError("kv: page_table must be [num_slots, max_pages], lengths [num_slots]")
        for name, t in (("page_table", page_table), ("lengths", lengths), ("counts", counts), ("stamps", stamps)):
            if t is not None and t.dtype != torch.int32:
                raise ValueError(f"kv: {name} must be int32")
        if counts is not None and counts.shape != lengths.shape:
            raise ValueError("kv: counts must be [num_slots]")
        if (weights is None) != (stamps is None):
            raise ValueError("kv: weights and stamps come together")
        if weights is not None and (weights.dtype != torch.float32 or weights.shape != k.shape[:3]
                                    or stamps.shape != k.shape[:3]):
            raise ValueError("kv: weights (float32) and stamps must be [num_pages, Hkv, page_size]")
        if any(t is not None and t.get_device() != k.get_device()
               for t in (v, page_table, lengths, counts, weights, stamps)):
            raise ValueError("kv: a cache's tensors lie on one device")
        self.k, self.v, self.page_table, self.lengths, self.counts = k, v, page_table, lengths, counts
        self.weights, self.stamps = weights, stamps
        self.dtype, self.Hkv, self.d, self.device = k.dtype, Hkv, d, k.get_device()
        self._c = kv_cache(k.data_ptr(), v.data_ptr(), DTYPE_CODE[k.dtype], Hkv, page_size, d, num_pages, *k_strides,
                           *v_strides, _ptr(page_table), page_table.shape[1], page_table.shape[0], _ptr(lengths),
                           _ptr(counts), _ptr(weights), _ptr(stamps))
        self._ref = C.byref(self._c)

    @classmethod
    def allocate(cls, num_pages, Hkv, page_size, d, num_slots, max_pages, dtype=torch.bfloat16,
                 weights=True, device="cuda") -> "KVCache":
        """Zeroed cache with an empty page table (-1); the caller hands out pages."""
        z = lambda shape, dt: torch.zeros(shape, dtype=dt, device=device)
        shape = (num_pages, Hkv, page_size)
        return cls(z(shape + (d,), dtype), z(shape + (d,), dtype), z((num_slots, max_pages), torch.int32).fill_(-1),
                   z((num_slots,), torch.int32), z((num_slots,), torch.int32),
                   z(shape, torch.float32) if weights else None, z(shape, torch.int32) if weights else None)

    @property
    def shape(self):
        return self.k.shape  # num_pages, Hkv, page_size, d


# A decode step's calls are short, and Python's part of them counts: the helpers below ask each tensor
# as little as the checks need (a call of kv_tree_attention took 21 us of the host's time, now 12).


def _rows(t: torch.Tensor, cache: KVCache, shape, name: str) -> kv_rows:
    strides = t.stride()
    if t.dtype is not cache.dtype or t.shape != shape or t.get_device() != cache.device or strides[3] != 1:
        raise ValueError(f"kv: {name} must be a tensor {list(shape)} of the cache's dtype on the cache's device, with "
                         "unit stride in d")
    return kv_rows(t.data_ptr(), strides[0], strides[1], strides[2])


def _ints(t, cache: KVCache, shape, name: str, dtype=torch.int32) -> int | None:
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.get_device() != cache.device or not t.is_contiguous():
        raise ValueError(f"kv: {name} must be a contiguous tensor of {dtype} and shape {list(shape)} on the cache's device")
    return t.data_ptr()


def _whole(t: torch.Tensor, cache: KVCache, name: str) -> int:
    if t.get_device() != cache.device or not t.is_contiguous():
        raise ValueError(f"kv: {name} must be a contiguous tensor on the cache's device")
    return t.data_ptr()


def _stream(stream, device: int) -> int:
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else _given_stream(stream)


def _on_device(cache: KVCache, fn, *args):
    """A call of the library, which takes the current device, on the cache's."""
    if torch._C._cuda_getDevice() == cache.device:
        return fn(*args)
    with torch.cuda.device(cache.device):
        return fn(*args)


def tree_masks(parents) -> torch.Tensor:
    """Mask words [B, T] (int64, on the CPU) of trees given by each node's parent: parents [B, T] with
    parents[b][i] < i, negative for a node that follows the cache directly."""
    parents = torch.as_tensor(parents).tolist()
    out = []
    for row in parents:
        words = []
        for i, p in enumerate(row):
            if p >= i:
                raise ValueError(f"kv: node {i} has parent {p}; a parent comes before its children")
            words.append((words[p] if p >= 0 else 0) | 1 << i)
        out.append([w - (1 << 64) if w >> 63 else w for w in words])
    return torch.tensor(out, dtype=torch.int64)


def _workspace(cache: KVCache, fn, *args) -> torch.Tensor:
    nbytes = _on_device(cache, fn, cache._ref, *args)
    if nbytes < 0:
        _check(int(nbytes))
    return torch.empty(max(16, nbytes), dtype=torch.uint8, device=cache.k.device)


def kv_tree_workspace(cache: KVCache, q) -> torch.Tensor:
    """Workspace for kv_tree_attention calls with queries of q's shape [B, T, Hq, d] (or a smaller batch)."""
    B, T, Hq = q.shape[:3]
    return _workspace(cache, lib().kv_tree_attention_workspace, B, T, Hq)


def kv_evict_workspace(cache: KVCache, B: int, budget: int) -> torch.Tensor:
    """Workspace for kv_evict calls of up to B sequences with this budget."""
    return _workspace(cache, lib().kv_evict_workspace, int(B), int(budget))


def kv_tree_attention(cache: KVCache, slots, q, k_new, v_new, mask, out, dev_err, workspace, num_nodes=None, lse=None,
                      scale=None, stream=None) -> None:
    """Attention of drafted nodes over the cache and one another: slots [B] int32; q [B, T, Hq, d];
    k_new, v_new [B, T, Hkv, d]; mask [B, T] int64 words (tree_masks); out [B, T, Hq, d]; lse None or
    [B, T, Hq] fp32; num_nodes None or [B] int32; workspace from kv_tree_workspace; dev_err [1] int32."""
    B, T, Hq, d = q.shape
    new = (B, T, cache.Hkv, d)
    rq, rk, rv = _rows(q, cache, q.shape, "q"), _rows(k_new, cache, new, "k_new"), _rows(v_new, cache, new, "v_new")
    if d != cache.d or out.shape != q.shape or out.dtype is not cache.dtype:
        raise ValueError("kv: q and out must be [B, T, Hq, d] of the cache's dtype and d")
    _check(_on_device(cache, lib().kv_tree_attention, cache._ref, B, T, Hq, _ints(slots, cache, (B,), "slots"), rq, rk, rv,
                      _ints(mask, cache, (B, T), "mask", torch.int64), _ints(num_nodes, cache, (B,), "num_nodes"),
                      1.0 / math.sqrt(d) if scale is None else scale, _whole(out, cache, "out"),
                      _ints(lse, cache, (B, T, Hq), "lse", torch.float32), _whole(workspace, cache, "workspace"),
                      workspace.numel(), _whole(dev_err, cache, "dev_err"), _stream(stream, cache.device)))


def kv_commit(cache: KVCache, slots, k_new, v_new, path, n_path, dev_err, stream=None) -> None:
    """Append the accepted path's keys and values: k_new, v_new [B, T, Hkv, d]; path [B, P] int32 node
    indices; n_path [B] int32."""
    B, T = k_new.shape[:2]
    P = path.shape[1]
    new = (B, T, cache.Hkv, cache.d)
    _check(_on_device(cache, lib().kv_commit, cache._ref, B, T, P, _ints(slots, cache, (B,), "slots"),
                      _rows(k_new, cache, new, "k_new"), _rows(v_new, cache, new, "v_new"),
                      _ints(path, cache, (B, P), "path"), _ints(n_path, cache, (B,), "n_path"),
                      _whole(dev_err, cache, "dev_err"), _stream(stream, cache.device)))


def kv_accumulate(cache: KVCache, slots, q, lse, path, n_path, dev_err, decay=1.0, scale=None, stream=None) -> None:
    """Add the accepted nodes' attention weights to the cache's entries, after kv_commit: q [B, T, Hq, d]
    and lse [B, T, Hq] of kv_tree_attention; path [B, P], n_path [B] int32 of kv_commit."""
    B, T, Hq, d = q.shape
    P = path.shape[1]
    if d != cache.d:
        raise ValueError("kv: q must have the cache's d")
    _check(_on_device(cache, lib().kv_accumulate, cache._ref, B, T, P, Hq, _ints(slots, cache, (B,), "slots"),
                      _rows(q, cache, q.shape, "q"), _ints(lse, cache, (B, T, Hq), "lse", torch.float32),
                      _ints(path, cache, (B, P), "path"), _ints(n_path, cache, (B,), "n_path"),
                      1.0 / math.sqrt(d) if scale is None else scale, decay, _whole(dev_err, cache, "dev_err"),
                      _stream(stream, cache.device)))


def kv_evict(cache: KVCache, slots, budget: int, recent: int, dev_err, workspace, stream=None) -> None:
    """Keep `budget` entries of each longer sequence, per key head: the `recent` newest tokens, then the
    largest weights. workspace from kv_evict_workspace."""
    B = slots.shape[0]
    _check(_on_device(cache, lib().kv_evict, cache._ref, B, _ints(slots, cache, (B,), "slots"), budget, recent,
                      _whole(workspace, cache, "workspace"), workspace.numel(), _whole(dev_err, cache, "dev_err"),
                      _stream(stream, cache.device)))


class Rotary:
    """Norms of queries and keys and the position rotation of an attention layer (kv_rotary in include/kv.h).

    inv_freq: radians a position of each turned pair (rot / 2 numbers, taken in 64 bits; their fractions of a
    turn are formed in doubles, off by 1.37 x 2^-53 of themselves at most: one radian a position is off by
    2^-36 turns at position 2^19, by 2^-24 at the end of the positions' type), or None for no rotation; axis:
    which of the `axes` positions each pair follows (None: the first); interleaved: pairs are neighbours, else
    elements i and i + rot / 2. q_norm, k_norm: None, or FP32 weights [d], or [heads, d] of each head, to which
    `offset` is added (1 for weights stored about zero).
    """

    def __init__(self, inv_freq=None, axis=None, axes: int = 1, interleaved: bool = False, q_norm=None, k_norm=None,
                 eps: float = 1e-6, offset: float = 0.0, device="cuda"):
        freq = [] if inv_freq is None else torch.as_tensor(inv_freq, dtype=torch.float64, device="cpu").tolist()
        if not all(math.isfinite(f) for f in freq):
            raise ValueError("kv: inv_freq must be finite")
        if axis is not None and (len(axis) != len(freq) or any(not 0 <= int(x) < axes for x in axis)):
            raise ValueError("kv: axis must name one of the axes for every frequency")
        if not 1 <= axes <= MAX_AXES:
            raise ValueError(f"kv: axes must be 1 to {MAX_AXES}")
        for name, t in (("q_norm", q_norm), ("k_norm", k_norm)):
            if t is not None and (t.dtype != torch.float32 or t.dim() not in (1, 2) or not t.is_cuda or t.stride(-1) != 1):
                raise ValueError(f"kv: {name} must be a float32 CUDA tensor [d] or [heads, d] with unit stride in d")
        norms = [t for t in (q_norm, k_norm) if t is not None]
        if norms:
            device = norms[0].device
        turns = [round(f / (2 * math.pi) * 2.0 ** 64) % (1 << 64) for f in freq]
        self.turns = torch.tensor([t - (1 << 64) if t >> 63 else t for t in turns], dtype=torch.int64, device=device)
        self.axis = None if axis is None else torch.tensor([int(x) for x in axis], dtype=torch.int32, device=device)
        self.q_norm, self.k_norm, self.rot, self.axes = q_norm, k_norm, 2 * len(freq), int(axes)
        self.device = self.turns.get_device()
        if any(t.get_device() != self.device for t in norms):
            raise ValueError("kv: the norms' weights lie on one device")
        head = lambda t: t.stride(0) if t is not None and t.dim() == 2 else 0
        at = lambda t: None if t is None else t.data_ptr()
        self._c = kv_rotary(at(q_norm), at(k_norm), head(q_norm), head(k_norm), eps, offset,
                            self.turns.data_ptr() if freq else None, at(self.axis), self.rot, self.axes, int(interleaved))
        self._ref = C.byref(self._c)

    def check(self, norm, heads: int, d: int) -> None:
        """That a side's weights are those of rows [heads, d]."""
        if norm is not None and norm.shape != (d,) and norm.shape != (heads, d):
            raise ValueError(f"kv: a norm's weights must be [{d}] or [{heads}, {d}]")


def _side(x, out, name: str, dtype, device: int, B: int, T: int, d: int):
    """kv_rows of a side of kv_norm_rotate [B, T, heads, d] and of its output, and its heads; nothing for neither."""
    if x is None and out is None:
        return None, None, 0
    if x is not None and out is not None and x.dim() == 4:
        shape, s, o = x.shape, x.stride(), out.stride()
        if shape[0] == B and shape[1] == T and shape[3] == d and out.shape == shape and x.dtype is dtype and \
                out.dtype is dtype and s[3] == 1 and o[3] == 1 and x.get_device() == device and out.get_device() == device:
            return kv_rows(x.data_ptr(), s[0], s[1], s[2]), kv_rows(out.data_ptr(), o[0], o[1], o[2]), shape[2]
    raise ValueError(f"kv: {name} and {name}_out must be tensors [B, T, heads, d] of one dtype on the rotary's device, with "
                     "unit stride in d")


def kv_norm_rotate(rotary: Rotary, positions, q=None, k=None, q_out=None, k_out=None, stream=None) -> None:
    """Norm and rotation of drafted tokens: q [B, T, Hq, d], k [B, T, Hkv, d] into q_out, k_out (which may be q
    and k); positions [axes, B, T] int32 ([B, T] with one axis; None where nothing is turned)."""
    like = q if q is not None else k
    if like is None or like.dim() != 4 or like.dtype not in DTYPE_CODE:
        raise ValueError("kv: q or k must be a tensor [B, T, heads, d] of a dtype of the cache's")
    device, dtype = rotary.device, like.dtype
    if device < 0:  # (tensors of the host would pass the checks of one device below)
        raise ValueError("kv: the rotary must lie on a CUDA device")
    B, T, _, d = like.shape
    rq, ro, Hq = _side(q, q_out, "q", dtype, device, B, T, d)
    rk, rp, Hkv = _side(k, k_out, "k", dtype, device, B, T, d)
    if rq is not None:
        rotary.check(rotary.q_norm, Hq, d)
    if rk is not None:
        rotary.check(rotary.k_norm, Hkv, d)
    shape = (B, T) if positions is not None and rotary.axes == 1 and positions.dim() == 2 else (rotary.axes, B, T)
    pos = _ints(positions, rotary, shape, "positions")
    _check(_on_device(rotary, lib().kv_norm_rotate, rotary._ref, DTYPE_CODE[dtype], B, T, Hq, Hkv, d, pos, rq, ro, rk, rp,
                      _stream(stream, device)))


def _packed(t, cache: KVCache, heads: int, total: int, name: str) -> kv_rows:
    s = t.stride()
    if t.shape != (total, heads, cache.d) or t.dtype is not cache.dtype or s[2] != 1 or t.get_device() != cache.device:
        raise ValueError(f"kv: {name} must be a tensor [{total}, {heads}, {cache.d}] of the cache's dtype on the cache's "
                         "device, with unit stride in d")
    return kv_rows(t.data_ptr(), 0, s[0], s[1])


def kv_append(cache: KVCache, slots, cu_seqlens, k, v, dev_err, rotary: Rotary | None = None, positions=None, q=None,
              q_out=None, stream=None) -> None:
    """The prompts' keys and values into the cache: k, v [total, Hkv, d], sequence b's rows cu_seqlens[b] on
    (cu_seqlens [B + 1] int32, on the device). With `rotary`, keys are normed and turned on the way, and q
    [total, Hq, d] into q_out (which may be q); positions [axes, total] int32 ([total] with one axis), None:
    the sequence's count and on. total may be 0."""
    B, total, Hkv, d, device = slots.shape[0], k.shape[0], cache.Hkv, cache.d, cache.device
    rk, rv = _packed(k, cache, Hkv, total, "k"), _packed(v, cache, Hkv, total, "v")
    rq = ro = ref = None
    Hq, axes = 0, 1
    if rotary is not None:
        if rotary.device != device:
            raise ValueError("kv: the rotary must lie on the cache's device")
        ref, axes = rotary._ref, rotary.axes
        rotary.check(rotary.k_norm, Hkv, d)
    if q is not None or q_out is not None:
        if q is None or q_out is None or rotary is None:
            raise ValueError("kv: q, q_out and rotary come together")
        Hq = q.shape[1]
        rq, ro = _packed(q, cache, Hq, total, "q"), _packed(q_out, cache, Hq, total, "q_out")
        rotary.check(rotary.q_norm, Hq, d)
    shape = (total,) if positions is not None and axes == 1 and positions.dim() == 1 else (axes, total)
    _check(_on_device(cache, lib().kv_append, cache._ref, B, total, Hq, _ints(slots, cache, (B,), "slots"),
                      _ints(cu_seqlens, cache, (B + 1,), "cu_seqlens"), rk, rv, ref,
                      _ints(positions, cache, shape, "positions"), rq, ro, _whole(dev_err, cache, "dev_err"),
                      _stream(stream, device)))


def kv_prompt_workspace(cache: KVCache, B: int, q) -> torch.Tensor:
    """Workspace for kv_prompt_attention calls of up to B sequences with queries of q's shape [total, Hq, d] (or
    fewer rows)."""
    return _workspace(cache, lib().kv_prompt_attention_workspace, int(B), q.shape[0], q.shape[1])


def kv_prompt_attention(cache: KVCache, slots, cu_seqlens, q, out, dev_err, workspace, lse=None, scale=None,
                        stream=None) -> None:
    """Causal attention of packed prompts over the cache, after kv_append of the same rows: q [total, Hq, d]; out
    [total, Hq, d]; lse None or [total, Hq] fp32; workspace from kv_prompt_workspace. total may be 0."""
    total, Hq = q.shape[:2]
    B = slots.shape[0]
    rq = _packed(q, cache, Hq, total, "q")
    if out.shape != q.shape or out.dtype is not cache.dtype:
        raise ValueError("kv: out must be [total, Hq, d] of the cache's dtype")
    _check(_on_device(cache, lib().kv_prompt_attention, cache._ref, B, total, Hq, _ints(slots, cache, (B,), "slots"),
                      _ints(cu_seqlens, cache, (B + 1,), "cu_seqlens"), rq,
                      1.0 / math.sqrt(cache.d) if scale is None else scale, _whole(out, cache, "out"),
                      _ints(lse, cache, (total, Hq), "lse", torch.float32), _whole(workspace, cache, "workspace"),
                      workspace.numel(), _whole(dev_err, cache, "dev_err"), _stream(stream, cache.device)))


def kv_fork(cache: KVCache, src, dst, new_pages, dev_err, stream=None) -> None:
    """Sequences dst become copies of sequences src ([n] int32 slots): page j is shared where new_pages[i][j]
    ([n, max_pages] int32) is negative, else copied to that page."""
    n = src.shape[0]
    _check(_on_device(cache, lib().kv_fork, cache._ref, n, _ints(src, cache, (n,), "src"), _ints(dst, cache, (n,), "dst"),
                      _ints(new_pages, cache, (n, cache.page_table.shape[1]), "new_pages"),
                      _whole(dev_err, cache, "dev_err"), _stream(stream, cache.device)))


def kv_compact_workspace(cache: KVCache) -> torch.Tensor:
    """Workspace for kv_compact calls."""
    return _workspace(cache, lib().kv_compact_workspace)


def kv_compact(cache: KVCache, used, dev_err, workspace, stream=None) -> None:
    """Moves the pages that sequences hold to the front of the pool; used [1] int32 takes their number (the pages
    from there on are free)."""
    _check(_on_device(cache, lib().kv_compact, cache._ref, _ints(used, cache, (1,), "used"),
                      _whole(workspace, cache, "workspace"), workspace.numel(), _whole(dev_err, cache, "dev_err"),
                      _stream(stream, cache.device)))
