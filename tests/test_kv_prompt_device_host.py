"""Host-only: a rotary whose tables lie in the host's memory is for looking at; its calls are refused, and no kernel gets
an address of the host."""
import pytest
import torch

from hybrid_ssm_gated_gb300 import kv


@pytest.fixture
def calls(monkeypatch):
    made = []

    class Library:
        def __getattr__(self, name):
            return lambda *args: made.append(name) or 0

    monkeypatch.setattr(kv, "lib", lambda: Library())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    return made


@pytest.mark.parametrize("freq", [None, [1.0, 0.5]], ids=["no turn", "turned"])
def test_host_tensors_are_refused(calls, freq):
    x = torch.zeros(2, 3, 4, 8)
    pos = torch.zeros(2, 3, dtype=torch.int32) if freq else None
    with pytest.raises(ValueError, match="CUDA"):
        kv.kv_norm_rotate(kv.Rotary(freq, device="cpu"), pos, q=x, q_out=torch.empty_like(x))
    assert not calls
