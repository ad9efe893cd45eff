"""The gated delta rule in chunks where a call makes several pairs of launches, which use two buffers in turn, and takes
a large batch in parts: against the same sequences resumed in calls of one pair each (which test_gpu_delta compares with
64 bits).  Both round alike; powers of two at the seams differ, 2^-18 of the state over all values."""
import pytest
import torch

from test_gpu_delta import inputs, near, run, ssd, to  # noqa: F401

pytestmark = pytest.mark.gpu


def chunk_bytes(B, H, G, N, dtype):
    """What the first launch leaves of 64 tokens (csrc/delta_chunk.cu)."""
    parts = 1 if dtype == torch.bfloat16 else 2
    return B * (H * ((2 * (N // 64) + parts) * 8192 + 5 * 64 * 4) + G * (N // 64) * 2 * 8192 * parts)


def chunks_of_a_pair(ssd, B, L, H, G, P, N, dtype):  # noqa: F811
    space, chunk = ssd.ssd_delta_workspace_size(B, L, H, P, N, dtype, G), chunk_bytes(B, H, G, N, dtype)
    if space == chunk * -(-L // 64):
        return -(-L // 64)
    return (space - B * H * P * N * 4) // (2 * chunk)


def in_pieces(ssd, A, O, lengths, piece, init):  # noqa: F811
    """y and the state after calls of at most `piece` tokens."""
    L, state, ys = A["x"].shape[1], init, []
    for lo in range(0, L, piece):
        part = {k: v[:, lo:lo + piece] if v.dim() > 1 else v for k, v in A.items()}
        y, state = ssd.ssd_delta_fwd(**part, **O, init_state=state, lengths=(lengths - lo).int())
        ys.append(y)
    return torch.cat(ys, 1), state


FORMS = [  # (heads, headdim): 16 columns a block, 32, and 32 with two blocks a multiprocessor (bf16)
    (8, 64), (40, 32), (80, 16)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("H,P", FORMS)
def test_several_pairs(ssd, H, P, N, dtype):  # noqa: F811
    """Four pairs or more; a sequence that ends in the first, one in the second, one in the last, and an idle one."""
    B, L = 4, 64
    while 3 * chunks_of_a_pair(ssd, B, L, H, H, P, N, dtype) * 64 >= L - 70:
        L += 640
    count = chunks_of_a_pair(ssd, B, L, H, H, P, N, dtype)
    assert -(-L // 64) > 3 * count
    a, o = inputs(B, L, H, H, P, N, dtype, seed=N + H)
    A, O = to(a), to(o)
    g = torch.Generator().manual_seed(1)
    cache = (torch.randn(6, H, P, N, generator=g) * 0.3).cuda()
    slots = torch.tensor([4, 1, 9, 2], dtype=torch.int32).cuda()
    lengths = torch.tensor([L - 5, count * 64 - 10, L, count * 64 + 700], dtype=torch.int32).cuda()
    final = torch.full_like(cache, 7.0)
    y, _ = ssd.ssd_delta_fwd(**A, **O, init_state=cache, slots=slots, lengths=lengths, final_state=final)
    rows = [0, 1, 3]
    alone = {k: v[rows] if v.dim() > 1 else v for k, v in A.items()}
    want_y, want = in_pieces(ssd, alone, O, lengths[rows], count * 64, cache[slots[rows].long()])
    near("final", final[slots[rows].long()], want.double().cpu(), 2.0 ** -18)
    near("y", y[rows], want_y.double().cpu(), 2.0 ** -18 if dtype == torch.float32 else 2.0 ** -7)
    assert not y[2].any() and (final[[0, 3, 5]] == 7.0).all()
    for b in range(B):
        assert not y[b, int(lengths[b]):].any()
    # in place, replayed, and again
    held = cache.clone()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        y2, _ = ssd.ssd_delta_fwd(**A, **O, init_state=held, slots=slots, lengths=lengths, final_state=held)
    for _ in range(6):
        held.copy_(cache)
        y2.fill_(float("nan"))
        graph.replay()
        assert torch.equal(y2, y) and torch.equal(held[slots[rows].long()], final[slots[rows].long()])
        assert torch.equal(held[[0, 3, 5]], cache[[0, 3, 5]])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cached", [False, True])
def test_a_batch_in_parts(ssd, cached, dtype):  # noqa: F811
    """So many heads that a part is one or two sequences, with and without rows of a cache; several pairs each."""
    B, L, H, P, N = 5, 3000, 160, 16, 128
    limit = 2 * (512 << 20) + 2 * H * P * N * 4
    assert ssd.ssd_delta_workspace_size(B, L, H, P, N, dtype, H) <= limit < 2 * 16 * chunk_bytes(B, H, H, N, dtype)
    a, o = inputs(B, L, H, H, P, N, dtype, seed=7)
    A, O = to(a), to(o)
    lengths = torch.tensor([L, 1500, L - 1, 0, L], dtype=torch.int32).cuda()
    g = torch.Generator().manual_seed(1)
    cache = (torch.randn(B + 2, H, P, N, generator=g) * 0.3).cuda()
    slots = torch.tensor([4, 1, 0, 6, 2], dtype=torch.int32).cuda() if cached else None
    rows = slots.long() if cached else torch.arange(B).cuda()
    positions = torch.tensor([3, 0, 9, 1, 0], dtype=torch.int32).cuda()
    final = torch.full_like(cache, 7.0)
    y, _ = ssd.ssd_delta_fwd(**A, **O, init_state=cache, slots=slots, lengths=lengths, positions=positions, final_state=final)
    init = cache[rows] * (positions > 0)[:, None, None, None]
    want_y, want = in_pieces(ssd, A, O, lengths, 320, init)
    near("final", final[rows], want.double().cpu(), 2.0 ** -18)
    near("y", y, want_y.double().cpu(), 2.0 ** -18 if dtype == torch.float32 else 2.0 ** -7)
    others = [i for i in range(B + 2) if i not in rows.tolist()]
    assert (final[others] == 7.0).all()
    held = cache.clone()
    for _ in range(6):  # in place
        held.copy_(cache)
        y2, _ = ssd.ssd_delta_fwd(**A, **O, init_state=held, slots=slots, lengths=lengths, positions=positions, final_state=held)
        assert torch.equal(y2, y) and torch.equal(held[rows], final[rows]) and torch.equal(held[others], cache[others])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,L,H,G,P,N", [(3, 150, 16, 8, 64, 64), (3, 150, 16, 8, 64, 128), (2, 90, 40, 20, 32, 128)])
def test_blocks_of_32_columns(ssd, B, L, H, G, P, N, dtype):  # noqa: F811
    """More blocks of 16 columns than multiprocessors, but not of 32: against 64 bits."""
    a, o = inputs(B, L, H, G, P, N, dtype, seed=L, cached=True)
    o["lengths"] = torch.tensor([L, 70, 1][:B], dtype=torch.int32)
    run(ssd, a, o)
