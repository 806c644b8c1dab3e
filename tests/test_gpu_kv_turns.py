"""Rotations at positions up to the ends of their type, against angles formed in whole numbers from pi itself."""
import math

import numpy as np
import pytest
import torch

from hybrid_ssm_gated_gb300 import build, kv
from tests.kv_ref import host
from tests.prompt_ref import turn_bound
from tests.turns_ref import angle, slack

pytestmark = pytest.mark.gpu

POSITIONS = [0, 1, -1, 77777, 2 ** 20 + 1, 10 ** 7 + 3, 2 ** 30 + 7, 2 ** 31 - 1, -2 ** 31]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    kv.lib()


@pytest.mark.parametrize("base", [1e4, 1e6])
@pytest.mark.parametrize("d,rot", [(128, 128), (80, 20)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions(base, d, rot, interleaved):
    T, h = len(POSITIONS), rot // 2
    freq = [base ** (-i / h) for i in range(h)]
    x = torch.from_numpy(np.random.default_rng(rot).normal(size=(1, T, 3, d))).float().cuda()
    out = torch.empty_like(x)
    pos = torch.tensor([POSITIONS], dtype=torch.int32, device="cuda")
    kv.kv_norm_rotate(kv.Rotary(freq, interleaved=interleaved), pos, q=x, q_out=out)
    y = host(x)[0]
    z, size, far = y.copy(), np.abs(y), np.zeros(y.shape)
    for i in range(h):
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
        a = np.array([angle(freq[i], t) for t in POSITIONS])[:, None]
        z[..., p], z[..., q] = y[..., p] * np.cos(a) - y[..., q] * np.sin(a), y[..., p] * np.sin(a) + y[..., q] * np.cos(a)
        size[..., p] = size[..., q] = np.abs(y[..., p]) + np.abs(y[..., q])
        # what the binding's fraction is off by, as often as the position says
        more = np.array([abs(t) * 2 * math.pi * float(slack(freq[i])) for t in POSITIONS])[:, None]
        far[..., p] = far[..., q] = size[..., p] * more
    off = np.abs(host(out)[0] - z)
    assert (off <= turn_bound(z, size, d, "f32") + far).all(), f"off by {off.max():.3e}"
