"""What the cache's tensor-core kernels leave when a wait runs out: an error bit, outputs as of refused
sequences, nothing read or written out of range, and a device that goes on.

Every wait of those kernels is bounded, by a second. The build for these tests (GDN_TEST_STALL) bounds them by
20 ms, and in one block of the grid lets a group of warps wait for an arrival that never comes; the block's other
warps then run out of theirs. Workspaces hold bytes that would be taken for the records of a call. The calls run in a
child process that loads that build through GDN_LIBRARY.
"""
import os
import subprocess
import sys

import numpy as np
import pytest

from hybrid_ssm_gated_gb300 import build, gdn
from tests import kv_stalled

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _both(call, name, tmp_path):
    """Results of the call with the normal library, and with the one whose waits run out."""
    build.build()
    env = dict(os.environ, GDN_LIBRARY=build.build(stall=True))
    r = subprocess.run([sys.executable, "-m", "tests.kv_stalled", call, name, str(tmp_path / "stalled.npz")], cwd=ROOT,
                       env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
    return kv_stalled.CALLS[call](name), dict(np.load(tmp_path / "stalled.npz"))


@pytest.mark.parametrize("name", kv_stalled.ATTENTION)
def test_attention_that_gives_up(name, tmp_path):
    """The units (sequence, key head) that the block had a part in are refused, the others to the bit."""
    want, got = _both("attention", name, tmp_path)
    assert want["err"] == 0 and got["err"] == gdn.DEVERR_TIMEOUT
    B, T, Hq, d = want["out"].shape
    heads = lambda x: x.reshape(B, T, 8, Hq // 8, -1).transpose(0, 2, 1, 3, 4).reshape(B * 8, -1)  # a row a unit
    same = (heads(got["out"]) == heads(want["out"])).all(1) & (heads(got["lse"]) == heads(want["lse"])).all(1)
    refused = (heads(got["out"]) == 0).all(1) & np.isneginf(heads(got["lse"])).all(1)
    assert (same | refused).all(), f"{(~(same | refused)).sum()} units are neither right nor refused"
    assert 1 <= refused.sum() <= 8


@pytest.mark.parametrize("name", kv_stalled.ACCUMULATION)
def test_accumulation_that_gives_up(name, tmp_path):
    """A weight is as it was, or the right one to the bit; of paths in two blocks of rows, or has gathered the
    first."""
    want, got = _both("accumulation", name, tmp_path)
    assert want["err"] == 0 and got["err"] == gdn.DEVERR_TIMEOUT
    before, w, new = got["before"], got["weights"], want["weights"]
    right = (w == new) | (w == before)
    if name == "two blocks of rows":
        right |= (w >= 0.5 * before) & (w <= new)
    assert np.array_equal(before, want["before"]) and right.all(), f"{(~right).sum()} weights are wrong"
    assert 64 <= ((w != new) & (new != before)).sum() <= 8 * 128 * 8
