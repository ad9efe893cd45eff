"""Sequences of the selective scan that two blocks share, where the state that
one hands to the other does not arrive."""
import pytest
import torch

import layer_ref as ref
from test_layer_cpu import SCAN_ARGS

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ssd():
    import mamba_ssd_forward_chunked_gb300 as m
    return m


# shared by blocks: more than four, and no more than seven, blocks of channels a multiprocessor
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("taken", [0, 1], ids=["lost", "taken"])
@pytest.mark.parametrize("in_place", [True, False], ids=["in-place", "apart"])
@pytest.mark.parametrize("B,L,C,N,lengths", [(2, 70, 5120, 16, None), (6, 100, 1700, 13, (0, 1, 100, 99, 50, 2)),
                                             (1, 130, 10001, 11, (33,))])
def test_a_block_takes_the_sequence_over(ssd, dtype, taken, in_place, B, L, C, N, lengths):
    g = torch.Generator().manual_seed(B + L + C)
    normal = lambda *s, dtype=F32: torch.randn(*s, generator=g).to(dtype).cuda()  # noqa: E731
    u, delta, z = (normal(B, L, C, dtype=dtype) for _ in range(3))
    Bm, Cm = normal(B, L, 1, N, dtype=dtype), normal(B, L, 1, N, dtype=dtype)
    A, D, bias, init = -torch.rand(C, N, generator=g).cuda() * N, normal(C), normal(C) - 2, normal(B, C, N)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    want = ssd.ssd_selective_scan(u, delta, A, Bm, Cm, D, z=z, delta_bias=bias, delta_softplus=True, init_state=init,
                                  lengths=n)
    bytes_ = ssd.ssd_selective_scan_workspace_size(B, L, C, N, 1)
    assert bytes_ > 0
    workspace = torch.zeros(bytes_, dtype=torch.uint8, device="cuda")
    y, state = torch.full_like(u, 9.0), init.clone()
    final = state if in_place else torch.full_like(init, 9.0)
    args = SCAN_ARGS.pack(SCAN_ARGS.size, B, L, C, N, 1, int(dtype == BF16), 1, 0,
                          *[t.data_ptr() for t in (u, delta, z, Bm, Cm)], *[L * C, C] * 3, *[L * N, N] * 2,
                          *[t.data_ptr() for t in (A, D, bias, state, final, y)], 0 if n is None else n.data_ptr(),
                          workspace.data_ptr(), bytes_)
    torch.cuda.synchronize()
    assert ssd.lib.ssd_debug_scan_handover(args, taken, None) == 0
    torch.cuda.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(final, want[1])
    if dtype == F32 and in_place and not taken:  # (what both agree on is right)
        r, e, h, eh = ref.scan(u, delta, A, Bm, Cm, D, z, bias, True, init, n)
        ref.check("y", y, r, ref.store(r, e, dtype))
        ref.check("state", final, h, eh + 2.0 ** -23 * h.abs() + 1e-30)
