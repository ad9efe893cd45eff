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
    """tensors(): two of the first device; the stream that is current is appended to `seen`."""
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

    def tensors():
        with FakeTensorMode():
            return torch.empty(4, 3, device="cuda:0"), torch.empty(2, 2, device="cuda:0")
    return tensors, seen


def test_a_stream_of_another_device_is_refused(ext, fake):
    tensors, seen = fake
    ran = []
    with pytest.raises(ext.SSDError, match="cuda:1.*cuda:0"):
        ext.layer._on(Stream(1), lambda *a: ran.append(a), None, *tensors())
    assert not ran and not seen
    with pytest.raises(ext.SSDError, match="cuda:1"):  # the states in a list, the parents beside it
        ext.layer._on(Stream(1), lambda *a: ran.append(a), [tensors()[0]], tensors()[1], None)
    assert not ran


def test_streams_are_those_of_the_tensors_device(ext, fake):
    tensors, seen = fake
    for stream in (Stream(0), 96, 0):
        assert ext.layer._on(stream, lambda *a: len(a), *tensors(), None) == 3
    assert seen == [(0, 64), (0, 96), (0, 0)]
