"""GPU parity of the cache operators of include/kv.h where their inputs or sizes are extreme: infinite keys
and rows without a log-sum-exp in the accumulation. References in 64 bits, as tests/test_gpu_kv.py.
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
