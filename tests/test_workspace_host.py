"""Whose scratch buffer a call gets (no GPU: the buffers lie in host memory, the stream and the
state of a capture are stand-ins)."""
import threading

import pytest
import torch

from log_space_sum_gb300 import api

DEV = torch.device("cpu")


@pytest.fixture
def at(monkeypatch):
    """The current stream and whether it is being captured."""
    now = {"stream": 1, "capturing": False}
    monkeypatch.setattr(api, "_stream", lambda device: now["stream"])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: now["capturing"])
    return now


def test_one_per_stream_reused_and_grown(at):
    a = api.workspace(1000, DEV)
    assert a.numel() >= 1000 and api.workspace(500, DEV) is a
    at["stream"] = 2
    assert api.workspace(500, DEV) is not a
    at["stream"] = 1
    assert api.workspace(500, DEV) is a
    assert api.workspace(5000, DEV).numel() >= 5000


def test_threads_on_one_stream_share_none(at):
    mine, theirs = api.workspace(1000, DEV), []
    thread = threading.Thread(target=lambda: theirs.append(api.workspace(1000, DEV)))
    thread.start()
    thread.join()
    assert theirs[0].data_ptr() != mine.data_ptr()
    assert api.workspace(1000, DEV) is mine


def test_a_captured_call_shares_none(at):
    eager = api.workspace(1000, DEV)
    at["capturing"] = True
    first, second = api.workspace(1000, DEV), api.workspace(1000, DEV)
    assert len({t.data_ptr() for t in (eager, first, second)}) == 3
    at["capturing"] = False
    # and the captured ones were not kept for later calls
    assert api.workspace(1000, DEV) is eager
