"""Which device and stream a Python call hands to the library, with the library and the CUDA runtime replaced by
records of the calls (no GPU)."""
import contextlib

import pytest
import torch

import gated_gqa_attention_gb300 as gda


class Workspace:
    """A tensor's face: 1024 bytes on cuda:1."""

    def data_ptr(self):
        return 4096

    def numel(self):
        return 1024

    def element_size(self):
        return 1

    def get_device(self):
        return 1


@pytest.fixture
def runtime(monkeypatch):
    """Two devices, cuda:0 current; device d's current stream is 100 + d."""
    state = {"device": 0, "calls": []}

    @contextlib.contextmanager
    def device(d):
        before, state["device"] = state["device"], d
        yield
        state["device"] = before

    class Library:
        def gda_workspace_init(self, *args):
            state["calls"].append((state["device"], args))
            return 0

    class Stream:
        cuda_stream = 100

    monkeypatch.setattr(gda, "load", lambda path=None: Library())
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: Stream())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state["device"], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 100 + d, raising=False)
    return state


def test_a_workspace_is_cleared_on_its_own_device(runtime):
    """In that device's current stream, where decode_ex on the same device follows it."""
    gda.workspace_init(Workspace())
    assert runtime["calls"] == [(1, (4096, 1024, 101))] and runtime["device"] == 0
