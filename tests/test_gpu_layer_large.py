"""Sizes at which the convolution's threads walk down more than one batch of
tokens, and the step's blocks take whole heads: the sizes of real prompts and
batches, which the small tests do not reach."""
import pytest
import torch

import layer_ref as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
both_types = pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])


@pytest.fixture(scope="module")
def ssd():
    import mamba_ssd_forward_chunked_gb300 as m
    return m


def blocks_of_eight(B, L, C):
    """The convolution's blocks if every thread took eight tokens (four channels each where they divide)."""
    return B * -(-(C // 4 if C % 4 == 0 else C) * -(-L // 8) // 128)


@both_types
@pytest.mark.parametrize("B,L,C,W,lengths", [
    (3, 1021, 2304, 4, (1021, 5, 181)),                           # runs of 24
    (3, 701, 1157, 3, (15, 701, 512)),                            # a channel at a time
    (3, 700, 2300, 2, None),
    (8, 2001, 4096, 4, (2001, 0, 1, 7, 130, 1000, 1999, 2000)),   # runs of over 100 tokens
])
def test_conv_runs(ssd, dtype, B, L, C, W, lengths):
    """Runs of several batches of eight tokens; sequences that end in the first, a middle and the last batch of a
    run; carried on from a ring, in rows of wider tensors."""
    per = 4 if dtype == F32 else 5  # blocks a multiprocessor holds
    assert blocks_of_eight(B, L, C) > per * torch.cuda.get_device_properties(0).multi_processor_count
    g = torch.Generator().manual_seed(B + L + C)
    normal = lambda *s, dtype=F32: torch.randn(*s, generator=g).to(dtype).cuda()  # noqa: E731
    u = normal(B, L, C + 16, dtype=dtype)[:, :, 8:8 + C]
    weight, bias, ring = normal(C, W), normal(C), normal(B, W, C, dtype=dtype)
    positions = torch.randint(0, 9, (B,), generator=g, dtype=torch.int32).cuda()
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    want, bound, after = ref.conv(u, weight, bias, ring, positions, n)
    split = (C - 300, 44, 256)
    new = torch.empty_like(ring)
    parts = ssd.ssd_conv_fwd(u, weight, bias, split=split, ring=ring, positions=positions, lengths=n, new_ring=new)
    for y, r, e in zip(parts, want.split(split, 2), bound.split(split, 2)):
        ref.check("y", y, r, ref.store(r, e, dtype))
    assert torch.equal(ref.d64(new), after)
    whole = ssd.ssd_conv_fwd(u, weight, bias, ring=ring, positions=positions, lengths=n)
    assert torch.equal(whole, torch.cat(parts, 2)) and torch.equal(ring, new)


@both_types
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("B,H,G,N", [(20, 16, 1, 64), (20, 16, 4, 128), (40, 8, 2, 256)])
def test_step_of_whole_heads(ssd, dtype, B, H, G, N, W):
    assert B * H >= 2 * torch.cuda.get_device_properties(0).multi_processor_count
    g = torch.Generator().manual_seed(B + H + N + W)
    normal = lambda *s, dtype=F32, scale=1.0: (torch.randn(*s, generator=g) * scale).to(dtype).cuda()  # noqa: E731
    C = H * 64 + 2 * G * N
    proj = normal(B, H * 64 + C + H, dtype=dtype)
    u, z, dt = proj[:, H * 64:H * 64 + C], proj[:, :H * 64], proj[:, H * 64 + C:]
    args = (u, dt, -torch.rand(H, generator=g).cuda() * 16, normal(H), normal(C, W, scale=0.5), normal(C, scale=0.5))
    state, ring = normal(B + 1, H, 64, N), normal(B + 1, W, C, dtype=dtype)
    positions = torch.randint(0, 9, (B,), generator=g, dtype=torch.int32).cuda()
    slots = torch.randperm(B + 1, generator=g)[:B].to(torch.int32)
    slots[3] = -1
    more = dict(ngroups=G, z=z, dt_bias=normal(H) - 3, slots=slots.cuda())
    y, by, h, eh, after = ref.step(*args, state, ring, positions, use_softplus=True, **more)
    new, kept = torch.full_like(state, 5.0), ring.clone()
    got = ssd.ssd_step(*args, state, kept, positions, dt_softplus=True, new_state=new, **more)
    ref.check("y", got, y, ref.store(y, by, dtype))
    live = [s for s in slots.tolist() if s >= 0]
    ref.check("state", new[live], h[live], eh[live] + 2.0 ** -23 * h[live].abs() + 1e-30)
    assert all((new[i] == 5.0).all() for i in range(B + 1) if i not in live)
    assert torch.equal(ref.d64(kept), after)
    ssd.ssd_step(*args, state, ring, positions, dt_softplus=True, **more)  # in place: the same bits
    assert torch.equal(state[live], new[live]) and torch.equal(ring, kept)
