"""The layer operators' `stream` argument."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def layer():
    from mamba_ssd_forward_chunked_gb300 import layer as m
    return m


def test_raw_handles(layer):
    """A raw handle is that stream; 0 is the default one, as for ssd_fwd."""
    side = torch.cuda.Stream()
    u = torch.zeros(1, 1, 8, device="cuda")
    with torch.cuda.stream(side):
        for handle in (0, side.cuda_stream, torch.cuda.default_stream(), side):
            got = layer._on(handle, lambda t: torch.cuda.current_stream().cuda_stream, u)
            assert got == getattr(handle, "cuda_stream", handle)
