"""Calls of the decay attention, the group norm and AdamW with tensors on another device than the current one are
refused on the host (no GPU work)."""
import pytest
import torch

from sub_linear_memory_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def library():
    build.build()


@pytest.mark.parametrize("module", ["decay", "norm", "optim"])
def test_tensors_elsewhere_are_refused(monkeypatch, module):
    from sub_linear_memory_gb300 import decay, norm, optim

    stream = {"decay": decay._stream, "norm": norm._stream, "optim": optim.AdamW._stream}[module]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    for device in ("cuda:1", "cpu"):
        with pytest.raises(ValueError, match="current CUDA device"):
            stream(torch.device(device))


def test_a_call_asks_for_its_device_before_all_else(monkeypatch):
    from sub_linear_memory_gb300 import decay

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    known = dict(decay._known)
    t = torch.zeros(4, 1, 64)
    for call in (lambda: decay.attn(t, t, t, torch.zeros(1)), lambda: decay.attn_bwd(t, t, t, torch.zeros(1), t),
                 lambda: decay.step(t, t, t, torch.zeros(1), torch.zeros(4, 1, 64, 64))):
        with pytest.raises(ValueError, match="current CUDA device"):
            call()
    assert decay._known == known
