"""The binding of the cache on a machine with several GPUs, with stand-ins for tensors and devices (no GPU
needed): calls and workspaces go to the cache's device, tensors of another are refused."""
import contextlib
import types

import pytest
import torch

from hybrid_ssm_gated_gb300 import kv


class Tensor:
    def __init__(self, shape, dtype, device):
        self.shape, self.dtype, self.device_index = torch.Size(shape), dtype, device

    def get_device(self):
        return self.device_index

    def stride(self):
        return torch.empty(self.shape, device="meta").stride()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096


CACHE = types.SimpleNamespace(device=1, dtype=torch.bfloat16, Hkv=2, d=8, _ref=None, k=torch.zeros(1))


@pytest.fixture
def current(monkeypatch):
    """The current device, 0 at first, as the binding asks for and changes it."""
    now = [0]

    @contextlib.contextmanager
    def device(i):
        old, now[0] = now[0], i
        yield
        now[0] = old

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now[0], raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    return now


def test_calls_run_on_the_device_of_the_cache(current):
    seen = []
    assert kv._on_device(CACHE, lambda *a: seen.append((current[0], a)) or 5, 1, 2) == 5
    assert seen == [(1, (1, 2))] and current == [0]
    current[0] = 1
    kv._on_device(CACHE, lambda: seen.append(current[0]))
    assert seen[-1] == 1 and current == [1]


def test_workspaces_are_asked_for_and_lie_there(current):
    asked = []
    ws = kv._workspace(CACHE, lambda ref, *a: asked.append((current[0], a)) or 100, 3, 4)
    assert asked == [(1, (3, 4))] and ws.numel() == 100 and ws.device == CACHE.k.device


@pytest.mark.parametrize("device", [-1, 0])
def test_tensors_of_another_device_are_refused(device):
    shape = (2, 3, 2, 8)
    kv._rows(Tensor(shape, torch.bfloat16, 1), CACHE, shape, "q")
    assert kv._ints(Tensor((2,), torch.int32, 1), CACHE, (2,), "slots") == 4096
    assert kv._whole(Tensor((1,), torch.int32, 1), CACHE, "dev_err") == 4096
    for call in (lambda: kv._rows(Tensor(shape, torch.bfloat16, device), CACHE, shape, "q"),
                 lambda: kv._ints(Tensor((2,), torch.int32, device), CACHE, (2,), "slots"),
                 lambda: kv._whole(Tensor((1,), torch.int32, device), CACHE, "dev_err")):
        with pytest.raises(ValueError, match="cache's device"):
            call()
