"""What names a device in the Python calls (no GPU: torch's queries are stand-ins)."""
import types

import pytest
import torch

import log_space_sum_gb300 as pc
from log_space_sum_gb300 import api


@pytest.fixture
def streams(monkeypatch):
    """Device 0 is current and its stream 70; device 1 has 71."""
    def current_stream(device=None):
        device = torch.device("cuda", device) if isinstance(device, int) else torch.device("cuda" if device is None else device)
        if device.type != "cuda":
            raise ValueError(f"Expected a cuda device, but got: {device}")
        return types.SimpleNamespace(cuda_stream=70 + (device.index or 0))

    monkeypatch.setattr(torch.cuda, "current_stream", current_stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 70 + index, raising=False)


@pytest.mark.parametrize("device,stream", [(0, 70), (1, 71), ("cuda", 70), ("cuda:1", 71), (torch.device("cuda"), 70),
                                           (torch.device("cuda:1"), 71), (torch.device("cuda", 0), 70)])
def test_every_name_of_a_device(streams, monkeypatch, device, stream):
    assert api._stream(device) == stream
    called = []
    monkeypatch.setattr(api.N, "call", lambda name, *args: called.append((name, *args)))
    pc.device_status(device)
    assert called == [("pc_device_status", stream)]


def test_none_and_the_wrong_device(streams, monkeypatch):
    called = []
    monkeypatch.setattr(api.N, "call", lambda name, *args: called.append((name, *args)))
    pc.device_status()
    pc.device_status(None)
    assert called == [("pc_device_status", 70)] * 2
    for device in ("cpu", torch.device("cpu")):
        with pytest.raises(ValueError, match="cuda device"):
            pc.device_status(device)
