"""The answering path's binding: what it needs of PyTorch when it is imported,
and whose workspace a call of attn_decode without one uses.  CPU only."""

import importlib.util

import pytest
import torch

from attention_backward_pass_attn_gb300 import binding as ab

NAMES = ("_cuda_getDevice", "_cuda_getCurrentRawStream", "_cuda_isCurrentStreamCapturing")


def test_import_needs_no_cuda_build(monkeypatch):
    """A PyTorch built without CUDA lacks these names."""
    for n in NAMES:
        monkeypatch.delattr(torch._C, n, raising=False)
    spec = importlib.util.spec_from_file_location(ab.__name__ + "_again", ab.__file__)
    mod = importlib.util.module_from_spec(spec)
    mod.__package__ = ab.__package__
    spec.loader.exec_module(mod)
    with pytest.raises(ValueError, match="CUDA tensor"):
        mod.rope_fwd(torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16), None, None, None)


class Streams:
    """Stands in for PyTorch's streams: the current one has a handle and an id."""

    def __init__(self, monkeypatch):
        self.handle, self.id, self.capturing, self.made = 0, 0, False, []
        monkeypatch.setattr(ab, "_decode_workspaces", {})
        monkeypatch.setattr(ab, "_current_stream", lambda dev: self.handle)
        monkeypatch.setattr(ab, "_capturing", lambda: self.capturing)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: self)
        monkeypatch.setattr(ab, "alloc_decode_workspace", lambda d, dev: self.make())
        monkeypatch.setattr(ab, "_empty", lambda *a: self.make())

    stream_id = property(lambda self: self.id)

    def make(self):
        self.made.append(object())
        return self.made[-1]

    def call(self, handle, sid, stream=None):
        self.handle, self.id = handle, sid
        return ab._decode_workspace(0, stream)[0]


@pytest.fixture
def streams(monkeypatch):
    class Library:
        @staticmethod
        def attn_decode_workspace_size(d):
            return 256
    monkeypatch.setattr(ab, "load_library", lambda: Library)
    return Streams(monkeypatch)


POOL = 0x7F0000001000  # a pool stream's handle; its id is a small number
EXTERNAL = 0x7F0000002000  # another owner's stream: its id is its handle


def test_workspaces_are_kept_for_streams_that_stay(streams):
    a = streams.call(0, 0)
    b = streams.call(POOL, 35)
    assert a is streams.call(0, 0) and b is streams.call(POOL, 35) and a is not b
    assert len(ab._decode_workspaces) == 2


def test_workspaces_are_not_kept_for_streams_that_may_go(streams):
    """A destroyed stream's handle may come back as another stream's while the
    first one's work still runs."""
    assert streams.call(EXTERNAL, EXTERNAL) is not streams.call(EXTERNAL, EXTERNAL)
    streams.capturing = True
    assert streams.call(POOL, 35) is not streams.call(POOL, 35)
    assert not ab._decode_workspaces


@pytest.mark.parametrize("stream", [None, 2])
def test_the_per_thread_stream_has_no_workspace(streams, stream):
    """Its handle is every thread's, the stream is not."""
    with pytest.raises(ValueError, match="workspace"):
        streams.call(2, 2, stream)
    assert not streams.made and not ab._decode_workspaces
