"""The layer operators on the GPU against 64-bit references (layer_ref.py),
with the error bounds stated there."""
import pytest
import torch

import layer_ref as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
IDS = {BF16: "bf16", F32: "f32"}
both_types = pytest.mark.parametrize("dtype", [BF16, F32], ids=IDS.get)


@pytest.fixture(scope="module")
def ssd():
    import mamba_ssd_forward_chunked_gb300 as m
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def ints(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def sliced(g, B, L, C, dtype, before=8, after=8):
    """Rows of C channels inside wider ones."""
    return normal(g, B, L, before + C + after, dtype=dtype)[:, :, before:before + C]


# ------------------------------------------------------------------ convolution

@both_types
@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("B,L,split,before", [
    (2, 1, (64, 16, 16), 8), (1, 2, (24,), 8), (2, 37, (264, 32, 32), 8), (1, 131, (100, 7), 3), (3, 70, (1,), 0),
    (1, 300, (1024, 128, 128), 16), (2, 33, (5, 3, 9), 1),
])
def test_conv_prompt(ssd, dtype, width, B, L, split, before):
    g = gen(B * 100 + L + width)
    C = sum(split)
    u = sliced(g, B, L, C, dtype, before=before)
    weight, bias = normal(g, C, width), normal(g, C)
    y = ssd.ssd_conv_fwd(u, weight, bias, split=split)
    want, bound, _ = ref.conv(u, weight, bias)
    for got, r, e in zip(y, want.split(split, 2), bound.split(split, 2)):
        assert got.is_contiguous()
        ref.check("y", got, r, ref.store(r, e, dtype))
    whole = ssd.ssd_conv_fwd(u, weight, None, activation=None)
    r, e, _ = ref.conv(u, weight, None, act=False)
    ref.check("no activation", whole, r, ref.store(r, e, dtype))


@both_types
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("width,C", [(4, 72), (3, 13), (2, 136)])
def test_conv_goes_on_from_its_ring(ssd, dtype, in_place, width, C):
    """Ragged pieces: lengths of zero, one and more than the ring; cache rows in
    another order; idle sequences; a fresh sequence over an uncleared row."""
    g = gen(width * 10 + C)
    B, L, S = 7, 67, 9
    u = sliced(g, B, L, C, dtype)
    weight, bias = normal(g, C, width), normal(g, C)
    ring = normal(g, S, width, C, dtype=dtype)
    ring[3] = float("nan")  # the row of a sequence at position 0
    positions, lengths = ints(5, 1, 0, 1000003, 2, 7, 0), ints(67, 0, 1, 2, 3, 40, 99)
    slots = ints(8, 0, 3, 5, 1, -1, 9)
    want, bound, after = ref.conv(u, weight, bias, ring, positions, lengths, slots)
    new = None if in_place else torch.full_like(ring, 77.0)
    before = ring.clone()
    y = ssd.ssd_conv_fwd(u, weight, bias, ring=ring, positions=positions, lengths=lengths, slots=slots, new_ring=new)
    ref.check("y", y, want, ref.store(want, bound, dtype))
    got = ring if in_place else new
    for row in range(S):
        if in_place or row in (8, 0, 3, 5, 1):
            assert torch.equal(torch.nan_to_num(ref.d64(got[row]), 55.0), torch.nan_to_num(after[row], 55.0)), row
        else:
            assert (got[row] == 77.0).all(), row
    if not in_place:
        assert torch.equal(torch.nan_to_num(ring), torch.nan_to_num(before))


@both_types
def test_conv_pieces_equal_the_whole(ssd, dtype):
    """A prompt in pieces, the last tokens one by one, is bit for bit the prompt at once."""
    g = gen(5)
    B, L, C, W = 2, 90, 320, 4
    u, weight, bias = normal(g, B, L, C, dtype=dtype), normal(g, C, W), normal(g, C)
    ring = torch.full((B, W, C), float("nan"), dtype=dtype, device="cuda")
    whole = ssd.ssd_conv_fwd(u, weight, bias)
    got, at = [], 0
    for n in (1, 2, 50, 3, 30, 1, 1, 1, 1):
        pos = torch.full((B,), at, dtype=torch.int32, device="cuda")
        got.append(ssd.ssd_conv_fwd(u[:, at:at + n], weight, bias, ring=ring, positions=pos))
        at += n
    assert at == L and torch.equal(torch.cat(got, 1), whole)


def test_conv_empty(ssd):
    w = torch.ones(8, 4, device="cuda")
    assert ssd.ssd_conv_fwd(torch.empty(0, 5, 8, device="cuda"), w).shape == (0, 5, 8)
    ring = torch.arange(64, dtype=F32, device="cuda").view(2, 4, 8)
    new = torch.zeros_like(ring)
    y = ssd.ssd_conv_fwd(torch.empty(2, 0, 8, device="cuda"), w, ring=ring, positions=ints(3, 4), new_ring=new)
    assert y.shape == (2, 0, 8) and torch.equal(new, ring)


# ------------------------------------------------------------------ selective scan

def scan_inputs(g, B, L, C, N, G, dtype):
    bc = normal(g, B, L, 2 * G * N + 8, dtype=dtype)
    return dict(u=sliced(g, B, L, C, dtype), delta=sliced(g, B, L, C, dtype), A=-torch.rand(C, N, generator=g).cuda() * N,
                Bm=bc[:, :, :G * N].unflatten(2, (G, N)), Cm=bc[:, :, G * N:2 * G * N].unflatten(2, (G, N)))


def check_scan(got, want, dtype):
    y, bound, h, eh = want
    ref.check("y", got[0], y, ref.store(y, bound, dtype))
    ref.check("state", got[1], h, eh + 2.0 ** -23 * h.abs() + 1e-30)


@both_types
@pytest.mark.parametrize("B,L,C,N,G", [
    (1, 1, 8, 16, 1), (3, 1, 130, 16, 1), (2, 5, 33, 1, 1), (1, 70, 96, 16, 3), (2, 129, 40, 13, 1), (1, 64, 64, 8, 2),
    (1, 33, 24, 32, 1), (1, 40, 17, 64, 1), (1, 700, 48, 16, 1), (2, 517, 8, 5, 1), (1, 260, 36, 33, 2),
    (1, 9001, 16, 16, 1), (1, 1300, 8, 40, 1),  # in 64 segments, the last of them empty; in ten
])
def test_scan(ssd, dtype, B, L, C, N, G):
    g = gen(B + 10 * L + C + N)
    s = scan_inputs(g, B, L, C, N, G, dtype)
    bare = ssd.ssd_selective_scan(s["u"], s["delta"].abs(), s["A"], s["Bm"], s["Cm"])
    check_scan(bare, ref.scan(s["u"], s["delta"].abs(), s["A"], s["Bm"], s["Cm"]), dtype)
    more = dict(D=normal(g, C), z=sliced(g, B, L, C, dtype), delta_bias=normal(g, C) - 2)
    init = normal(g, B, C, N)
    got = ssd.ssd_selective_scan(**s, **more, delta_softplus=True, init_state=init)
    check_scan(got, ref.scan(**s, **more, use_softplus=True, init=init), dtype)


@both_types
@pytest.mark.parametrize("L,C,N", [(1, 40, 16), (300, 40, 16), (1100, 16, 7)])
def test_scan_lengths_and_in_place(ssd, dtype, L, C, N):
    """Sequences of every length from none to all; what lies after a sequence's
    end (here NaN) changes nothing; the state is updated where it is."""
    g = gen(L)
    B = 6
    s = scan_inputs(g, B, L, C, N, 1, dtype)
    lengths = ints(0, 1, L, max(0, L - 1), L // 2, min(2, L))
    for b in range(B):
        for k in ("u", "delta", "Bm", "Cm"):
            s[k][b, int(lengths[b]):] = float("nan")
    z = sliced(g, B, L, C, dtype)
    state = normal(g, B, C, N)
    init = state.clone()
    y, h = ssd.ssd_selective_scan(**s, z=z, delta_softplus=True, init_state=state, final_state=state, lengths=lengths)
    assert h is state
    clean = {k: torch.nan_to_num(v) if k != "A" else v for k, v in s.items()}
    check_scan((y, h), ref.scan(**clean, z=z, use_softplus=True, init=init, lengths=lengths), dtype)
    for b in range(B):
        assert (y[b, int(lengths[b]):] == 0).all()
    assert torch.equal(state[0], init[0])


@both_types
@pytest.mark.parametrize("B,L,C,N,G", [(2, 70, 5120, 16, 1), (1, 100, 10001, 11, 1), (3, 65, 3400, 13, 2), (1, 33, 9800, 16, 1)])
def test_scan_blocks_share_sequences(ssd, dtype, B, L, C, N, G):
    """More blocks of channels than the GPU holds in even numbers: blocks take
    equal runs of tokens, and hand over the states where a run ends inside a
    sequence.  Again with the same workspace, whatever it holds."""
    g = gen(B + L + C)
    s = scan_inputs(g, B, L, C, N, G, dtype)
    more = dict(D=normal(g, C), z=sliced(g, B, L, C, dtype), delta_bias=normal(g, C) - 2, init_state=normal(g, B, C, N))
    want = ref.scan(**s, **{k: v for k, v in more.items() if k != "init_state"}, use_softplus=True, init=more["init_state"])
    got = ssd.ssd_selective_scan(**s, **more, delta_softplus=True)
    check_scan(got, want, dtype)
    workspace = torch.full((ssd.ssd_selective_scan_workspace_size(B, L, C, N, G),), 1, dtype=torch.uint8, device="cuda")
    assert workspace.numel() > 0
    for _ in range(2):
        again = ssd.ssd_selective_scan(**s, **more, delta_softplus=True, workspace=workspace)
        assert all(torch.equal(x, y) for x, y in zip(again, got))


@both_types
def test_scan_blocks_share_sequences_in_place(ssd, dtype):
    g = gen(8)
    B, L, C, N = 6, 100, 1700, 16
    s = scan_inputs(g, B, L, C, N, 1, dtype)
    lengths = ints(0, 1, L, L - 1, L // 2, 2)
    state = normal(g, B, C, N)
    init = state.clone()
    y, h = ssd.ssd_selective_scan(**s, delta_softplus=True, init_state=state, final_state=state, lengths=lengths)
    check_scan((y, h), ref.scan(**s, use_softplus=True, init=init, lengths=lengths), dtype)
    for b in range(B):
        assert (y[b, int(lengths[b]):] == 0).all()
    assert torch.equal(state[0], init[0])


def test_scan_extremes(ssd):
    """Steps of zero, decays that vanish and states that never fade."""
    g = gen(8)
    s = scan_inputs(g, 1, 600, 32, 16, 1, F32)
    s["delta"] = s["delta"].abs()
    s["delta"][:, ::7] = 0.0
    s["delta"][:, 3::50] = 80.0
    s["A"][:8] = 0.0
    s["A"][8:16] = -1000.0
    got = ssd.ssd_selective_scan(**s)
    check_scan(got, ref.scan(**s), F32)


@pytest.mark.parametrize("L", [1, 37, 1000])
def test_scan_steps_of_zero_keep_the_state(ssd, L):
    g = gen(11)
    s = scan_inputs(g, 2, L, 48, 16, 1, F32)
    s["delta"] = torch.zeros_like(s["delta"])
    init = normal(g, 2, 48, 16)
    _, h = ssd.ssd_selective_scan(**s, init_state=init)
    assert torch.equal(h, init)
    s["delta"], s["u"], s["A"] = s["delta"] + 1.0, torch.zeros_like(s["u"]), torch.zeros_like(s["A"])  # and no decay
    _, h = ssd.ssd_selective_scan(**s, init_state=init)
    assert torch.equal(h, init)


def test_scan_pieces_and_single_tokens(ssd):
    """A prompt, then tokens one at a time from its state, as the whole at once."""
    g = gen(9)
    B, L, C, N = 2, 530, 72, 16
    s = scan_inputs(g, B, L, C, N, 1, F32)
    want = ref.scan(**s, use_softplus=True)
    state, got = None, []
    for a, b in ((0, 520), (520, 521), (521, 529), (529, 530)):
        part = {k: v if k == "A" else v[:, a:b] for k, v in s.items()}
        y, state = ssd.ssd_selective_scan(**part, delta_softplus=True, init_state=state)
        got.append(y)
    check_scan((torch.cat(got, 1), state), want, F32)


def test_scan_empty(ssd):
    e = torch.empty(2, 0, 8, device="cuda")
    bc = torch.empty(2, 0, 1, 4, device="cuda")
    init = torch.randn(2, 8, 4, device="cuda")
    y, h = ssd.ssd_selective_scan(e, e, torch.ones(8, 4, device="cuda"), bc, bc, init_state=init)
    assert y.shape == (2, 0, 8) and torch.equal(h, init)
    _, h = ssd.ssd_selective_scan(e, e, torch.ones(8, 4, device="cuda"), bc, bc)
    assert (h == 0).all()
    _, h = ssd.ssd_selective_scan(e[:0], e[:0], torch.ones(8, 4, device="cuda"), bc[:0], bc[:0])
    assert h.shape == (0, 8, 4)


# ------------------------------------------------------------------ single token

@both_types
@pytest.mark.parametrize("B,H,G,N,W", [(1, 4, 1, 128, 4), (3, 6, 2, 64, 4), (5, 4, 4, 256, 3), (2, 3, 1, 64, 2),
                                       (40, 16, 1, 128, 4)])
def test_step(ssd, dtype, B, H, G, N, W):
    g = gen(B + H + N)
    C = H * 64 + 2 * G * N
    pad = 1 if B == 3 else 0  # rows that are not 16-byte aligned
    proj = normal(g, B, H * 64 + C + H + pad, dtype=dtype)
    u, z, dt = proj[:, H * 64:H * 64 + C], proj[:, :H * 64], proj[:, H * 64 + C:H * 64 + C + H]
    A, D, dt_bias = -torch.rand(H, generator=g).cuda() * 16, normal(g, H), normal(g, H) - 3
    weight, bias = normal(g, C, W, scale=0.5), normal(g, C, scale=0.5)
    state, ring = normal(g, B + 2, H, 64, N), normal(g, B + 2, W, C, dtype=dtype)
    positions = torch.randint(0, 9, (B,), generator=g, dtype=torch.int32).cuda()
    slots = torch.randperm(B + 2, generator=g)[:B].to(torch.int32)
    if B > 2:
        slots[1] = -1
    slots = slots.cuda()
    args = (u, dt, A, D, weight, bias)
    more = dict(ngroups=G, z=z, dt_bias=dt_bias, slots=slots)
    y, by, h, eh, after = ref.step(*args, state, ring, positions, use_softplus=True, **more)
    new = torch.full_like(state, 5.0)
    ring2 = ring.clone()
    got = ssd.ssd_step(*args, state, ring2, positions, dt_softplus=True, new_state=new, **more)
    ref.check("y", got, y, ref.store(y, by, dtype))
    live = [int(s) for s in slots if s >= 0]
    ref.check("state", new[live], h[live], eh[live] + 2.0 ** -23 * h[live].abs() + 1e-30)
    assert all((new[i] == 5.0).all() for i in range(B + 2) if i not in live)
    assert torch.equal(ref.d64(ring2), after)
    ssd.ssd_step(*args, state, ring, positions, dt_softplus=True, **more)  # in place: the same bits
    assert torch.equal(state[live], new[live]) and torch.equal(ring, ring2)


def test_step_plain_options(ssd):
    """No gate, no biases, dt as given in 32 bits beside bfloat16."""
    g = gen(1)
    B, H, N, W = 2, 2, 64, 4
    C = H * 64 + 2 * N
    u, dt = normal(g, B, C, dtype=BF16), torch.rand(B, H, generator=g).cuda() * 0.1
    A, D, weight = -torch.ones(H).cuda(), normal(g, H), normal(g, C, W)
    state, ring, pos = normal(g, B, H, 64, N), normal(g, B, W, C, dtype=BF16), ints(0, 2)
    y, by, h, eh, _ = ref.step(u, dt, A, D, weight, None, state, ring, pos, 1)
    got = ssd.ssd_step(u, dt, A, D, weight, None, state, ring, pos)
    ref.check("y", got, y, ref.store(y, by, BF16))
    ref.check("state", state, h, eh + 2.0 ** -23 * h.abs() + 1e-30)


def test_step_continues_a_prompt(ssd):
    """conv + ssd_fwd over a prompt, then ssd_step token by token, against the
    recurrence over all tokens (the prompt's own tolerance: 5e-3 of the largest
    value, as in the parity tests)."""
    g = gen(4)
    B, L, T, H, G, N, W = 2, 150, 6, 4, 1, 64, 4
    C = H * 64 + 2 * G * N
    u = normal(g, B, L + T, C)
    dt = torch.rand(B, L + T, H, generator=g).cuda() * 0.1
    A, D, weight, bias = -torch.rand(H, generator=g).cuda() * 8, normal(g, H), normal(g, C, W, scale=0.5), normal(g, C)
    ring = torch.zeros(B, W, C, device="cuda")
    x, Bm, Cm = ssd.ssd_conv_fwd(u[:, :L], weight, bias, split=(H * 64, G * N, G * N), ring=ring)
    y, state = ssd.ssd_fwd(x.view(B, L, H, 64), dt[:, :L].contiguous(), A, Bm.view(B, L, G, N), Cm.view(B, L, G, N), D, 64)
    outs = [y]
    for t in range(L, L + T):
        pos = torch.full((B,), t, dtype=torch.int32, device="cuda")
        outs.append(ssd.ssd_step(u[:, t], dt[:, t], A, D, weight, bias, state, ring, pos)[:, None])
    got = torch.cat(outs, 1).double().cpu()
    r, _, _ = ref.conv(u, weight, bias)
    x, Bm, Cm = r[..., :H * 64].view(B, -1, H, 64), r[..., H * 64:H * 64 + N], r[..., H * 64 + N:]
    h, want = torch.zeros(B, H, 64, N, dtype=torch.float64), []
    d, A, D = ref.d64(dt), ref.d64(A), ref.d64(D)
    for t in range(L + T):
        dx = (d[:, t, :, None] * x[:, t])[..., None]
        h = torch.exp(d[:, t] * A)[..., None, None] * h + dx * Bm[:, t, None, None]
        want.append((h * Cm[:, t, None, None]).sum(-1) + D[:, None] * x[:, t])
    want = torch.stack(want, 1)
    assert float((got - want).abs().max()) <= 5e-3 * float(want.abs().max())
    assert float((state.double().cpu() - h).abs().max()) <= 5e-3 * float(h.abs().max())


def test_step_cache_past_32_bit_offsets(ssd):
    """A row whose first element lies beyond 2^31 elements of the cache."""
    H, N, W = 16, 256, 4
    S = 2 ** 31 // (H * 64 * N) + 3
    C = H * 64 + 2 * N
    g = gen(6)
    state = torch.zeros(S, H, 64, N, device="cuda")
    ring = torch.zeros(S, W, C, device="cuda")
    row = S - 1
    state[row] = normal(g, H, 64, N)
    u, dt, pos = normal(g, 1, C), torch.rand(1, H, generator=g).cuda(), ints(0)
    A, D, weight = -torch.ones(H).cuda(), normal(g, H), normal(g, C, W)
    y, by, h, eh, _ = ref.step(u, dt, A, D, weight, None, state[row:], ring[row:], pos, 1)
    got = ssd.ssd_step(u, dt, A, D, weight, None, state, ring, pos, slots=ints(row))
    ref.check("y", got, y, ref.store(y, by, F32))
    ref.check("state", state[row:], h, eh + 2.0 ** -23 * h.abs() + 1e-30)
    assert (state[:row].amax() == 0) and torch.equal(ring[row, 0], u[0])


# ------------------------------------------------------------------ 4-bit weights

@both_types
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,n,k", [(1, 16, 64), (1, 1, 1), (2, 50, 200), (3, 33, 129), (8, 48, 320), (9, 20, 65),
                                   (17, 130, 1000), (1, 700, 2048), (16, 64, 640), (5, 17, 63), (40, 16, 96),
                                   (9, 9731, 257), (16, 9760, 128)])  # two row tiles a block
def test_w4(ssd, dtype, group, M, n, k):
    g = gen(M * 7 + n + k + group)
    codes = torch.randint(0, 16, (n, k), generator=g)
    packed, scales = ssd.w4_pack(codes.cuda()), torch.rand(n, -(-k // group), generator=g).cuda() + 0.5
    x = normal(g, M, k + 8, dtype=dtype)[:, 3:3 + k] if M == 3 else normal(g, M, k, dtype=dtype)
    add = normal(g, M, n + 5, dtype=dtype)[:, 1:1 + n]
    for a in (None, add):
        want, bound = ref.w4(x, codes, scales, group, a)
        ref.check("y", ssd.ssd_w4_matvec(x, packed, scales, group, add=a), want, ref.store(want, bound, dtype))


@pytest.mark.parametrize("dtype,top", [(BF16, 8), (F32, 2 ** 13)], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,n,k,group", [(1, 96, 1024, 128), (3, 40, 777, 32), (8, 33, 512, 64), (12, 16, 130, 128)])
def test_w4_whole_numbers_are_exact(ssd, dtype, top, M, n, k, group):
    """Whole numbers whose sums stay below 2^24 (and, in bfloat16, are written
    to 32 bits' worth of powers of two): every product has to be right."""
    g = gen(k)
    codes = torch.randint(0, 16, (n, k), generator=g)
    x = torch.randint(-top // 8, top // 8 + 1, (M, k), generator=g).to(dtype).cuda()
    scales = (2.0 ** torch.randint(0, 2, (n, -(-k // group)), generator=g)).cuda()
    y = ssd.ssd_w4_matvec(x, ssd.w4_pack(codes).cuda(), scales, group)
    want, _ = ref.w4(x, codes, scales, group)
    assert float(want.abs().max()) < 2 ** 24
    assert torch.equal(ref.d64(y), ref.d64(want.to(dtype)))


def test_w4_keeps_other_tokens_apart(ssd):
    """Infinities and NaN of one token stay with it; codes and activations past
    the matrix's edges do not exist."""
    g = gen(2)
    codes = torch.randint(0, 16, (20, 70), generator=g)
    packed, scales = ssd.w4_pack(codes).cuda(), torch.ones(20, 3, device="cuda")
    wide = torch.full((4, 100), float("nan"), device="cuda")
    wide[:, :70] = normal(g, 4, 70)
    clean = ssd.ssd_w4_matvec(wide[:, :70], packed, scales, 32)
    assert torch.isfinite(clean).all()
    wide[1, 5], wide[2, 69] = float("inf"), float("nan")
    y = ssd.ssd_w4_matvec(wide[:, :70], packed, scales, 32)
    assert torch.equal(y[0], clean[0]) and torch.equal(y[3], clean[3])
    assert torch.isnan(y[2]).all() and not torch.isfinite(y[1, codes[:, 5].cuda() != 8]).any()


def test_w4_quantized_product(ssd):
    g = gen(12)
    w, x = normal(g, 100, 300), normal(g, 2, 300)
    packed, scales = ssd.w4_quantize(w, 64)
    y = ssd.ssd_w4_matvec(x, packed, scales, 64)
    want = ref.d64(x) @ ref.d64(w).t()
    step = ref.d64(scales).repeat_interleave(64, 1)[:, :300]
    assert ((ref.d64(y) - want).abs() <= 0.51 * (ref.d64(x).abs() @ step.t()) + 1e-4).all()


# ------------------------------------------------------------------ beam search

def same_choice(got, want, where=""):
    best, parents, tokens = got
    r, rp, rt = want
    assert torch.equal(parents.cpu().long(), rp), where
    assert torch.equal(tokens.cpu().long(), rt), where
    fine = torch.isfinite(r)
    assert torch.equal(torch.isfinite(best.cpu()), fine)
    # the log-sum-exp and two additions: EPS of each term
    assert ((ref.d64(best) - r).abs()[fine] <= ref.EPS * (r.abs()[fine] + 32)).all()


@both_types
@pytest.mark.parametrize("B,W,V,k", [(1, 1, 5, 5), (2, 4, 1000, 4), (1, 8, 32001, 16), (3, 3, 77, 64), (1, 2, 20000, 1),
                                     (2, 5, 4099, 10), (1, 64, 300, 64), (40, 2, 9001, 4)])
def test_beam_select(ssd, dtype, B, W, V, k):
    g = gen(V + k)
    # ties within a beam (bfloat16 logits repeat) but, by the beams' irregular scores, not between beams
    logits = normal(g, B, W, V + 3, dtype=dtype, scale=3.0)[:, :, 1:V + 1]
    scores = (-30 * torch.rand(B, W, generator=g)).cuda()
    finished = (torch.rand(B, W, generator=g) < 0.3).cuda()
    same_choice(ssd.ssd_beam_select(logits, scores, k), ref.beam(logits, scores, k))
    same_choice(ssd.ssd_beam_select(logits, scores, k, finished=finished, eos=V - 1),
                ref.beam(logits, scores, k, finished, V - 1))


@both_types
def test_beam_ties_and_masks(ssd, dtype):
    """Equal logits, beams that are copies, masked tokens, rows with nothing
    left, beams at minus infinity, NaN and infinite logits."""
    inf = float("inf")
    x = torch.zeros(8, 4, 5000, dtype=dtype)
    s = torch.tensor([-1.0, -1.0, -inf, -2.0]).repeat(8, 1)
    x[1, :, 1000:] = -inf                       # most of the vocabulary masked
    x[2] = -inf                                 # nothing left anywhere
    x[3, 0] = -inf                              # nothing left in the best beam
    x[4, :, 4990:] = 3.0                        # the best at the end, many of them
    x[5, 0, 17] = float("nan")                  # a beam that is lost
    x[6, 1, 40] = inf                           # likewise
    x[7] = torch.finfo(dtype).min               # the type's lowest value everywhere, as some masks have it
    x[7, :, 123] = 0.0
    x[7, :, 124] = 0.0
    for k in (1, 4, 37, 64):
        same_choice(ssd.ssd_beam_select(x.cuda(), s.cuda(), k), ref.beam(x, s, k), k)
    done = torch.tensor([True, False, True, False]).repeat(8, 1)
    for eos in (0, 4999):
        same_choice(ssd.ssd_beam_select(x.cuda(), s.cuda(), 8, finished=done.cuda(), eos=eos), ref.beam(x, s, 8, done, eos))


@both_types
def test_beam_low_logits_beside_masked_ones(ssd, dtype):
    """Logits far below 0 beside whole stretches of minus infinity or of the
    type's lowest value: the sums must neither overflow nor lose them."""
    g = gen(31)
    V = 40000
    x = (torch.randn(4, 3, V, generator=g) - 1000.0).to(dtype)
    x[1, :, 100:39000] = -float("inf")
    x[2, :, 100:39000] = torch.finfo(dtype).min
    x[3, 1:] = torch.finfo(dtype).min
    s = torch.tensor([-1.0, -2.5, -4.0]).repeat(4, 1)
    for k in (1, 6):
        same_choice(ssd.ssd_beam_select(x.cuda(), s.cuda(), k), ref.beam(x, s, k), k)


@both_types
def test_beam_many_requests_of_ties(ssd, dtype):
    """Enough rows for the long pieces, with ties, masks and finished beams."""
    g = gen(32)
    x = (torch.randint(0, 4, (40, 4, 70000), generator=g)).to(dtype)
    x[::3] = 0.0
    x[1::3, :, :69990] = -float("inf")
    s = torch.tensor([-1.0, -1.0, -1.5, -9.0]).repeat(40, 1)
    done = torch.zeros(40, 4, dtype=torch.bool)
    done[5:9, 1] = True
    done[7] = True
    # equal sums in every beam of a request whose rows are equal
    x[:, 1] = x[:, 0]
    for k in (4, 64):
        same_choice(ssd.ssd_beam_select(x.cuda(), s.cuda(), k, finished=done.cuda(), eos=69999),
                    ref.beam(x, s, k, done, 69999), k)


def test_beam_scores_that_swallow_small_differences(ssd):
    """A beam at -2^23 (units of 1): logits that differ by less are equal scores,
    and fall by index, not by logit.  All beams share one row, hence one sum."""
    g = gen(77)
    row = torch.randn(30000, generator=g)
    row[29000] = 9.0
    x = row.expand(1, 2, -1).contiguous().cuda()
    s = torch.full((1, 2), -2.0 ** 23).cuda()
    best, parents, tokens = ssd.ssd_beam_select(x, s, 12)
    lse = torch.logsumexp(row.double(), 0)
    score = (torch.tensor(-2.0 ** 23) + (row - lse.float())).view(1, -1).expand(2, -1).reshape(-1)
    want = score.sort(descending=True, stable=True)[1][:12]
    # no candidate lies so near half a unit that a rounding of the sum could move its score
    assert (((row.double() - lse) % 1.0 - 0.5).abs()[row > 1.0] > 1e-5).all()
    assert torch.equal(parents.cpu().long()[0] * 30000 + tokens.cpu().long()[0], want)
    assert torch.equal(best.cpu()[0], score[want])


@pytest.mark.parametrize("beams,rows,dtype", [(4, (6, 64), F32), (3, (7,), BF16), (1, (5,), torch.uint8),
                                              (8, (3, 3), torch.uint8), (64, (16,), F32), (17, (33, 4), F32)])
def test_reorder(ssd, beams, rows, dtype):
    g = gen(beams)
    B = 5
    states = [(torch.rand(B * beams, *rows, generator=g) * 200).to(dtype).cuda(),
              torch.randn(B * beams, 128, generator=g).cuda()]
    parents = torch.randint(0, beams, (B, beams), generator=g, dtype=torch.int32)
    parents[0] = torch.arange(beams)             # nothing moves
    parents[1] = torch.arange(beams).flip(0)     # everything does
    parents[2] = 0
    at = (torch.arange(B)[:, None] * beams + parents).view(-1).cuda()
    want = [t[at] for t in states]
    new = ssd.ssd_beam_reorder(states, parents.cuda(), out=[torch.zeros_like(t) for t in states])
    assert all(torch.equal(a, b) for a, b in zip(new, want))
    ssd.ssd_beam_reorder(states, parents.cuda())
    assert all(torch.equal(a, b) for a, b in zip(states, want))


def test_reorder_other_counts_and_bad_parents(ssd):
    src = torch.arange(24, dtype=F32, device="cuda").view(6, 4)
    out = torch.full((10, 4), -1.0, device="cuda")
    parents = torch.tensor([[2, 0, 3, 1, 1], [-1, 1, 0, 99, 2]], dtype=torch.int32).cuda()
    ssd.ssd_beam_reorder([src], parents, out=[out])
    for b in range(2):
        for i, p in enumerate(parents[b].tolist()):
            assert torch.equal(out[b * 5 + i], src[b * 3 + p] if 0 <= p < 3 else torch.full((4,), -1.0).cuda()), (b, i)
    many = [torch.randn(6, 3 + i, device="cuda") for i in range(20)]
    par = ints(1, 1, 0, 2, 0, 2).view(2, 3)
    want = [t[torch.tensor([1, 1, 0, 5, 3, 5]).cuda()] for t in many]
    ssd.ssd_beam_reorder(many, par)
    assert all(torch.equal(a, b) for a, b in zip(many, want))
    assert ssd.ssd_beam_reorder([], par) == []


# ------------------------------------------------------------------ offsets past 32 bits

def far_apart(g, rows, C, dtype, L=None):
    """[rows, L, C] (or [rows, C]) whose rows lie 2^31 + 64 elements apart."""
    gap = 2 ** 31 + 64
    shape, stride = ((rows, L, C), (gap, C + 8, 1)) if L else ((rows, C), (gap, 1))
    t = torch.empty(gap * (rows - 1) + (L or 1) * (C + 8), dtype=dtype, device="cuda").as_strided(shape, stride)
    return t.copy_(normal(g, *shape, dtype=dtype))


def test_inputs_far_apart(ssd):
    g = gen(41)
    u = far_apart(g, 2, 40, BF16, L=11)
    weight = normal(g, 40, 4)
    y, e, _ = ref.conv(u, weight, None)
    ref.check("conv", ssd.ssd_conv_fwd(u, weight), y, ref.store(y, e, BF16))
    s = scan_inputs(g, 2, 11, 40, 16, 1, BF16)
    s["u"] = u
    check_scan(ssd.ssd_selective_scan(**s, delta_softplus=True), ref.scan(**s, use_softplus=True), BF16)
    one = {k: v if k == "A" else v[:, :1] for k, v in s.items()}
    check_scan(ssd.ssd_selective_scan(**one, delta_softplus=True), ref.scan(**one, use_softplus=True), BF16)
    del u, s, one
    x = far_apart(g, 2, 96, BF16)
    codes = torch.randint(0, 16, (40, 96), generator=g)
    scales = torch.rand(40, 3, generator=g).cuda()
    y, e = ref.w4(x, codes, scales, 32)
    ref.check("w4", ssd.ssd_w4_matvec(x, ssd.w4_pack(codes).cuda(), scales, 32), y, ref.store(y, e, BF16))
    del x
    logits = far_apart(g, 2, 300, BF16)[None]
    scores = normal(g, 1, 2)
    same_choice(ssd.ssd_beam_select(logits, scores, 5), ref.beam(logits, scores, 5))


def test_reorder_of_rows_past_32_bits(ssd):
    row = 2 ** 31 + 48
    t = torch.empty(2, row, dtype=torch.uint8, device="cuda")
    t[0], t[1] = 3, 7
    t[0, -1], t[1, -1], t[0, 5] = 11, 13, 17
    ssd.ssd_beam_reorder([t], ints(1, 0).view(1, 2))
    assert int(t[0, -1]) == 13 and int(t[1, -1]) == 11 and int(t[1, 5]) == 17 and int(t[0, 5]) == 7
    assert int(t[0, :-1].min()) == 7 == int(t[0, :-1].max())


# ------------------------------------------------------------------ streams, repeats, refusals

def test_other_stream_and_repeats(ssd):
    """On a stream of its own each call gives what it gives on the default one,
    bit for bit, however often it runs."""
    g = gen(21)
    B, L, C = 2, 400, 256
    u, weight = normal(g, B, L, C, dtype=BF16), normal(g, C, 4)
    s = scan_inputs(g, B, L, C, 16, 1, BF16)
    x, codes = normal(g, 4, 640, dtype=BF16), torch.randint(0, 16, (100, 640), generator=g)
    packed, scales = ssd.w4_pack(codes).cuda(), torch.rand(100, 5, generator=g).cuda()
    logits, scores = normal(g, B, 4, 30000), normal(g, B, 4)

    def once(**kw):
        return [ssd.ssd_conv_fwd(u, weight, **kw), *ssd.ssd_selective_scan(**s, delta_softplus=True, **kw),
                ssd.ssd_w4_matvec(x, packed, scales, 128, **kw), *ssd.ssd_beam_select(logits, scores, 8, **kw)]
    want = once()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream):
        for _ in range(3):
            got = once() if stream is None else once(stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_decoding_step_in_a_cuda_graph(ssd):
    """One token's calls captured once and replayed on other inputs give what
    the calls give outside (states, rings and choices bit for bit)."""
    g = gen(51)
    B, W, H, N, V = 2, 3, 4, 64, 500
    C, rows = H * 64 + 2 * N, B * W
    u, dt, pos = normal(g, rows, C, dtype=BF16), torch.rand(rows, H, generator=g).cuda(), ints(*range(rows))
    A, D, weight = -torch.rand(H, generator=g).cuda(), normal(g, H), normal(g, C, 4)
    state, ring = normal(g, rows, H, 64, N), normal(g, rows, 4, C, dtype=BF16)
    packed = ssd.w4_pack(torch.randint(0, 16, (V, H * 64), generator=g)).cuda()
    scales, scores = torch.rand(V, 4, generator=g).cuda() * 0.1, normal(g, B, W)

    def token():
        y = ssd.ssd_step(u, dt, A, D, weight, None, state, ring, pos)
        logits = ssd.ssd_w4_matvec(y.view(rows, -1), packed, scales, 64)
        best, parents, tokens = ssd.ssd_beam_select(logits.view(B, W, V), scores, W)
        ssd.ssd_beam_reorder([state, ring], parents)
        return best, parents, tokens
    keep = [t.clone() for t in (state, ring)]
    token()
    for t, k in zip((state, ring), keep):
        t.copy_(k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            out = token()
    torch.cuda.current_stream().wait_stream(side)
    for seed in (1, 2):
        u.copy_(normal(gen(seed), rows, C, dtype=BF16))
        for t, k in zip((state, ring), keep):
            t.copy_(k)
        want = [t.clone() for t in token()] + [state.clone(), ring.clone()]
        for t, k in zip((state, ring), keep):
            t.copy_(k)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip([*out, state, ring], want))


def test_refusals(ssd):
    z = lambda *shape, dtype=F32: torch.zeros(*shape, dtype=dtype, device="cuda")  # noqa: E731
    E = ssd.SSDError
    u, w = z(2, 5, 12), z(12, 4)
    for bad in (dict(weight=z(12, 5)), dict(weight=z(11, 4)), dict(weight=w.cpu()), dict(weight=w.to(BF16)),
                dict(bias=z(11)), dict(split=(4, 4)), dict(split=(4, 4, 2, 2)), dict(split=(12, 0)),
                dict(activation="relu"), dict(ring=z(2, 3, 12)), dict(ring=z(2, 4, 12, dtype=BF16)),
                dict(slots=ints(0, 1)), dict(new_ring=z(2, 4, 12)), dict(ring=z(1, 4, 12)), dict(lengths=ints(1)),
                dict(positions=torch.zeros(2, device="cuda")), dict(out=z(2, 5, 11)), dict(u=z(2, 5, 24)[:, :, ::2]),
                dict(u=z(2, 5, 12, dtype=torch.float16)), dict(u=z(5, 12))):
        with pytest.raises(E):
            ssd.ssd_conv_fwd(**{"u": u, "weight": w, **bad})
    scan = dict(u=u, delta=u, A=z(12, 16), Bm=z(2, 5, 1, 16), Cm=z(2, 5, 1, 16))
    for bad in (dict(delta=u.to(BF16)), dict(delta=z(2, 4, 12)), dict(A=z(12, 8)), dict(Bm=z(2, 5, 16)),
                dict(Bm=z(2, 5, 1, 65), Cm=z(2, 5, 1, 65), A=z(12, 65)), dict(Bm=z(2, 5, 5, 16), Cm=z(2, 5, 5, 16)),
                dict(D=z(3)), dict(z=z(2, 5, 13)), dict(init_state=z(2, 12, 8)), dict(final_state=z(1, 12, 16)),
                dict(lengths=z(2)), dict(y=z(2, 5, 12, dtype=BF16)),
                dict(Bm=z(2, 5, 2, 32)[..., :16], Cm=z(2, 5, 2, 16))):
        with pytest.raises(E):
            ssd.ssd_selective_scan(**{**scan, **bad})
    step = dict(u=z(2, 384), dt=z(2, 4), A=z(4), D=z(4), weight=z(384, 4), bias=None, state=z(2, 4, 64, 64),
                ring=z(2, 4, 384), positions=ints(0, 0))
    ssd.ssd_step(**step)
    for bad in (dict(u=z(2, 385)), dict(dt=z(2, 3)), dict(dt=z(2, 4, dtype=BF16)), dict(ngroups=2), dict(ngroups=0),
                dict(A=z(5)), dict(D=None), dict(weight=z(384, 1)), dict(state=z(2, 4, 64, 64, dtype=BF16)),
                dict(state=z(1, 4, 64, 64), ring=z(1, 4, 384)), dict(ring=z(3, 4, 384)), dict(positions=None),
                dict(slots=ints(0)), dict(z=z(2, 255)), dict(new_state=z(3, 4, 64, 64)), dict(y=z(2, 4, 63)),
                dict(state=z(2, 4, 32, 64), u=z(2, 256), weight=z(256, 4), ring=z(2, 4, 256))):
        with pytest.raises(E):
            ssd.ssd_step(**{**step, **bad})
    w4 = dict(x=z(2, 100), packed=z(2, 2, 32, 4, dtype=torch.int32), scales=z(20, 4), group=32)
    ssd.ssd_w4_matvec(**w4)
    for bad in (dict(x=z(2, 129)), dict(group=33), dict(group=64), dict(scales=z(40, 4)), dict(packed=z(2, 2, 32, 4)),
                dict(add=z(2, 21)), dict(add=z(2, 20, dtype=BF16)), dict(y=z(1, 20))):
        with pytest.raises(E):
            ssd.ssd_w4_matvec(**{**w4, **bad})
    sel = dict(logits=z(2, 4, 50), scores=z(2, 4), k=4)
    for bad in (dict(k=0), dict(k=65), dict(logits=z(2, 1, 3), scores=z(2, 1)), dict(scores=z(2, 3)),
                dict(finished=z(2, 4)), dict(finished=z(2, 4) > 0), dict(finished=z(2, 4) > 0, eos=50),
                dict(workspace=z(1, dtype=torch.uint8)), dict(logits=z(2, 4, 100)[:, :, ::2])):
        with pytest.raises(E):
            ssd.ssd_beam_select(**{**sel, **bad})
    par = ints(0, 0, 1, 1).view(2, 2)
    for bad in (dict(states=[z(5, 4)]), dict(states=[z(4, 4), z(6, 4)]), dict(states=[z(6, 4)]), dict(states=[z(4, 4).cpu()]),
                dict(states=[z(4, 8)[:, ::2]]), dict(states=[z(4, 4)], out=[]), dict(states=[z(4, 4)], out=[z(5, 4)]),
                dict(states=[z(4, 4)], parents=par.long()), dict(states=[z(4, 4)], parents=par.cpu())):
        with pytest.raises(E):
            ssd.ssd_beam_reorder(**{"parents": par, **bad})
