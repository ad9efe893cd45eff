"""The layer operators' `stream` argument, without a GPU: tensors that have a
device but no memory, and streams that only have a name."""
import contextlib

import pytest
import torch

try:
    from torch._subclasses.fake_tensor import FakeTensorMode
except ImportError:
    FakeTensorMode = None


@pytest.fixture(scope="module")
def ext():
    import __graft_entry__
    __graft_entry__.build()
    import mamba_ssd_forward_chunked_gb300 as m
    return m


class Stream:
    def __init__(self, index, handle=64):
        self.device, self.cuda_stream = torch.device("cuda", index), handle


@pytest.fixture
def fake(monkeypatch):
    """tensors(index): two of that device; the stream that is current is appended to `seen`."""
    if FakeTensorMode is None:
        pytest.skip("no tensors without memory")
    seen = []

    @contextlib.contextmanager
    def current(stream):
        seen.append((stream.device.index, stream.cuda_stream))
        yield
    monkeypatch.setattr(torch.cuda, "stream", current)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: Stream(torch.device(device).index, handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(torch.device(device).index, 0))

    def tensors(index):
        with FakeTensorMode():
            return torch.empty(4, 3, device=f"cuda:{index}"), torch.empty(2, 2, device=f"cuda:{index}")
    return tensors, seen


def test_a_stream_of_another_device_is_refused(ext, fake):
    tensors, seen = fake
    ran = []
    with pytest.raises(ext.SSDError, match="cuda:0.*cuda:1"):
        ext.layer._on(Stream(0), lambda *a: ran.append(a), None, *tensors(1))
    assert not ran and not seen
    with pytest.raises(ext.SSDError, match="cuda:0"):  # the states in a list, the parents beside it
        ext.layer._on(Stream(0), lambda *a: ran.append(a), [tensors(1)[0]], tensors(1)[1], None)
    assert not ran


def test_streams_are_those_of_the_tensors_device(ext, fake):
    tensors, seen = fake
    for stream in (Stream(1), 96, 0):
        assert ext.layer._on(stream, lambda *a: len(a), *tensors(1), None) == 3
    assert seen == [(1, 64), (1, 96), (1, 0)]
