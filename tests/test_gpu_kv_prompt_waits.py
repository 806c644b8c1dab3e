"""What the prompt attention on the tensor cores leaves when a wait runs out: an error bit, rows as of refused sequences,
nothing read or written out of range, and a device that goes on (as tests/test_gpu_kv_waits.py, whose build of the
library it uses)."""
import os
import subprocess
import sys

import numpy as np
import pytest

from hybrid_ssm_gated_gb300 import build, gdn
from tests import prompt_stalled

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("name", prompt_stalled.CALLS)
def test_attention_that_gives_up(name, tmp_path):
    """The rows that the block had a part in are refused, the others to the bit."""
    build.build()
    env = dict(os.environ, GDN_LIBRARY=build.build(stall=True))
    r = subprocess.run([sys.executable, "-m", "tests.prompt_stalled", name, str(tmp_path / "stalled.npz")], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
    want, got = prompt_stalled.call(name), dict(np.load(tmp_path / "stalled.npz"))
    assert want["err"] == 0 and got["err"] == gdn.DEVERR_TIMEOUT
    same = (got["out"] == want["out"]).all(2) & (got["lse"] == want["lse"])
    refused = (got["out"] == 0).all(2) & np.isneginf(got["lse"])
    assert (same | refused).all(), f"{(~(same | refused)).sum()} rows are neither right nor refused"
    assert refused.any() and refused.mean() < 0.5
