"""Calls with tensors on another device than the current one are refused on the
host (no GPU work)."""
import pytest
import torch

from sub_linear_memory_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def library():
    build.build()


@pytest.mark.parametrize("module", ["binding", "q8"])
def test_tensors_elsewhere_are_refused(monkeypatch, module):
    """The stream that a call launches on is asked for by the tensors' device,
    before anything is launched."""
    from sub_linear_memory_gb300 import binding, q8

    stream = {"binding": binding, "q8": q8}[module]._stream
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    for device in ("cuda:1", "cpu"):
        with pytest.raises(ValueError, match="current CUDA device"):
            stream(torch.device(device))


def test_the_current_device_is_taken(monkeypatch):
    from sub_linear_memory_gb300 import binding

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    binding.check_device(torch.device("cuda:3"))
