"""Calls of the C entry points from several host threads."""
import ctypes
import threading

import pytest
import torch

from test_layer_cpu import SELECT_ARGS

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ssd():
    import mamba_ssd_forward_chunked_gb300 as m
    return m


def test_beam_selections_of_two_threads(ssd):
    """Two widths whose blocks take different amounts of shared memory, each from
    a thread and on a stream of its own (ctypes lets go of the interpreter)."""
    B, W, V = 10, 64, 64  # rows enough for the long pieces
    logits, scores = torch.randn(B, W, V, device="cuda"), torch.randn(B, W, device="cuda")
    codes, keep = {}, []

    def calls(k):
        stream = torch.cuda.Stream()
        n = ssd.ssd_beam_select_workspace_size(B, W, V, k)
        out = [torch.empty(n, dtype=torch.uint8, device="cuda")] + [torch.empty(B, k, dtype=torch.int32, device="cuda") for _ in range(3)]
        keep.append((stream, out))
        args = ctypes.create_string_buffer(SELECT_ARGS.pack(
            SELECT_ARGS.size, B, W, V, k, 0, -1, 0, logits.data_ptr(), W * V, V, scores.data_ptr(), 0,
            *[t.data_ptr() for t in out[1:]], out[0].data_ptr(), n), SELECT_ARGS.size)

        def loop():
            codes[k] = {ssd.lib.ssd_beam_select(args, stream.cuda_stream) for _ in range(6000)}
        return threading.Thread(target=loop)
    torch.cuda.synchronize()
    threads = [calls(63), calls(64)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == {63: {0}, 64: {0}}
