"""Convolution, delta rule and verification together, as a model with drafted
tokens uses them; captured, on other streams, with offsets past 32 bits."""
import pytest
import torch

import delta_ref as ref
from test_gpu_delta import NORM, inputs, near, to

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ssd():
    import mamba_ssd_forward_chunked_gb300 as m
    return m


class Model:
    """One layer: embedding, convolution of x | B | C, delta rule, output."""

    def __init__(self, ssd, H=4, G=2, P=64, N=128, V=97, dtype=torch.float32):
        g = torch.Generator().manual_seed(1)
        rand = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
        self.ssd, self.H, self.G, self.P, self.N, self.V, self.dtype = ssd, H, G, P, N, V, dtype
        self.split = (H * P, G * N, G * N)
        C = sum(self.split)
        self.embed, self.gates = rand(V, C).to(dtype), rand(V, 2 * H).to(dtype)
        self.weight, self.bias, self.out = rand(C, 4) * 0.4, rand(C) * 0.1, rand(H * P, V) * 20.0
        self.A, self.dt_bias = -torch.exp(rand(H)), rand(H) - 3.0

    def caches(self, slots):
        C = sum(self.split)
        return (torch.full((slots, 4, C), 3.0, device="cuda", dtype=self.dtype),
                torch.full((slots, self.H, self.P, self.N), 3.0, device="cuda"))

    def __call__(self, tokens, ring, state, slots, positions, lengths=None, keep=True):
        """Logits; the caches go on by ``lengths`` tokens, or stay without ``keep``."""
        B, L = tokens.shape
        u, gates = self.embed[tokens.long()], self.gates[tokens.long()]
        x, Bm, Cm = self.ssd.ssd_conv_fwd(u, self.weight, self.bias, split=self.split, ring=ring, positions=positions,
                                          lengths=lengths, slots=slots, new_ring=None if keep else torch.empty_like(ring))
        y, _ = self.ssd.ssd_delta_fwd(x.view(B, L, self.H, self.P), gates[..., :self.H], self.A, Bm.view(B, L, self.G, self.N),
                                      Cm.view(B, L, self.G, self.N), gates[..., self.H:], dt_bias=self.dt_bias,
                                      dt_softplus=True, beta_sigmoid=True, norm_eps=NORM, init_state=state, slots=slots,
                                      positions=positions, lengths=lengths, final_state=state if keep else None,
                                      want_final_state=keep)
        return torch.matmul(y.reshape(B, L, -1).float(), self.out)


@pytest.mark.parametrize("L", [1, 9, 70])
def test_drafts_are_verified_and_committed(ssd, L):
    """Drafts of several rounds; afterwards every sequence's caches are those of its tokens one by one."""
    model, B, T = Model(ssd), 5, 4
    g = torch.Generator().manual_seed(L)
    slots = torch.tensor([6, 0, 3, 2, 5], dtype=torch.int32).cuda()
    ring, state = model.caches(7)
    prompt = torch.randint(0, model.V, (B, L), generator=g).cuda()
    lengths = torch.tensor([L, 1, L, max(1, L - 1), L], dtype=torch.int32).cuda()
    positions = torch.zeros(B, dtype=torch.int32).cuda()
    logits = model(prompt, ring, state, slots, positions, lengths)
    last = logits[torch.arange(B), lengths.long() - 1].argmax(-1)
    sequences = [prompt[b, :int(lengths[b])].tolist() for b in range(B)]
    positions = lengths.clone()
    counts = []
    for _ in range(6):
        draft = torch.randint(0, model.V, (B, T), generator=g).int().cuda()
        now = torch.cat([last[:, None].int(), draft], 1)
        logits = model(now, ring, state, slots, positions, keep=False)
        draft[:, 0] = torch.where(torch.rand(B, generator=g).cuda() < 0.7, logits[:, 0].argmax(-1).int(), draft[:, 0])
        now[:, 1] = draft[:, 0]
        logits = model(now, ring, state, slots, positions, keep=False)
        tokens, accepted, logprobs = ssd.ssd_draft_verify(logits, draft, torch.rand(B, T + 1, generator=g).cuda())
        want = torch.log_softmax(logits.double(), -1).gather(2, tokens.clamp(min=0).long()[..., None])[..., 0]
        assert ((logprobs - want).abs()[tokens >= 0] < 2.0 ** -16).all()
        counts += accepted.tolist()
        model(now, ring, state, slots, positions, accepted + 1)
        for b in range(B):
            n = int(accepted[b])
            sequences[b] += now[b, :n + 1].tolist()
            assert torch.equal(tokens[b, :n], draft[b, :n])
            last[b] = tokens[b, n]
        positions = positions + accepted + 1
    assert len(set(counts)) > 1  # some were accepted, some not
    ring2, state2 = model.caches(7)
    for b in range(B):
        for t, token in enumerate(sequences[b]):
            model(torch.tensor([[token]]).cuda(), ring2, state2, slots[b:b + 1], torch.tensor([t], dtype=torch.int32).cuda())
    assert torch.equal(ring[slots.long()], ring2[slots.long()])
    near("states", state[slots.long()], state2[slots.long()].double().cpu(), 2.0 ** -18)
    assert (state[[1, 4]] == 3.0).all() and (ring[[1, 4]] == 3.0).all()


def test_rounds_in_a_cuda_graph(ssd):
    """A prompt in chunks, a verification and the commitment, captured once and replayed on other inputs."""
    a, o = inputs(2, 150, 4, 2, 64, 128, torch.bfloat16, seed=1)
    A, O = to(a), to(o)
    logits, draft = torch.randn(2, 4, 500, device="cuda"), torch.randint(0, 500, (2, 3), device="cuda", dtype=torch.int32)
    u = torch.rand(2, 4, device="cuda")
    state = torch.zeros(2, 4, 64, 128, device="cuda")
    steps = {k: v[:, :4].clone() if v.dim() > 1 else v for k, v in A.items()}

    def round_():
        y, final = ssd.ssd_delta_fwd(**A, **O, final_state=state)
        tokens, accepted, _ = ssd.ssd_draft_verify(logits, draft, u)
        y2, _ = ssd.ssd_delta_fwd(**steps, **O, init_state=state, final_state=state, lengths=accepted + 1)
        return y, tokens, accepted, y2
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        round_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = round_()
    torch.cuda.current_stream().wait_stream(side)
    for seed in range(3):
        g = torch.Generator().manual_seed(seed)
        logits.copy_(torch.randn(2, 4, 500, generator=g) * 4)
        draft.copy_(logits[:, :3].argmax(-1))
        u.copy_(torch.rand(2, 4, generator=g))
        A["x"].copy_(torch.randn(A["x"].shape, generator=g))
        graph.replay()
        held, s = [v.clone() for v in got], state.clone()
        want = round_()
        assert all(torch.equal(v, w) for v, w in zip(held, want)) and torch.equal(s, state)


def test_streams_side_by_side(ssd):
    """Calls on two streams at once, each with its own workspace, are those of one."""
    jobs = []
    for seed, (B, L, H) in enumerate(((2, 700, 4), (3, 333, 8))):
        a, o = inputs(B, L, H, H, 128, 128, torch.bfloat16, seed=seed)
        jobs.append((to(a), to(o), torch.randn(8, 6, 5000, device="cuda"), torch.randint(0, 5000, (8, 5), device="cuda", dtype=torch.int32),
                     torch.rand(8, 6, device="cuda")))

    def call(job, **more):
        return [*ssd.ssd_delta_fwd(**job[0], **job[1], **more), *ssd.ssd_draft_verify(*job[2:], **more)]
    want = [call(j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [[call(j, stream=s) for j, s in zip(jobs, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(v, w) for turn in got for one, two in zip(turn, want) for v, w in zip(one, two))


def test_given_workspaces(ssd):
    a, o = inputs(1, 100, 2, 1, 64, 128, torch.bfloat16)
    A, O = to(a), to(o)
    n = ssd.ssd_delta_workspace_size(1, 100, 2, 64, 128, torch.bfloat16)
    assert n > 0 and ssd.ssd_delta_workspace_size(1, 5, 2, 64, 128, torch.bfloat16) == 0
    want = ssd.ssd_delta_fwd(**A, **O)
    space = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert torch.equal(ssd.ssd_delta_fwd(**A, **O, workspace=space)[0], want[0])
    with pytest.raises(ssd.SSDError):
        ssd.ssd_delta_fwd(**A, **O, workspace=space[:-16])
    with pytest.raises(ssd.SSDError):
        ssd.ssd_delta_fwd(**A, **O, workspace=space[4:])
    v = torch.randn(1, 2, 50, device="cuda"), torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.rand(1, 2, device="cuda")
    n = ssd.ssd_draft_verify_workspace_size(1, 1, 50, torch.float32, False)
    assert torch.equal(ssd.ssd_draft_verify(*v, workspace=torch.empty(n, dtype=torch.uint8, device="cuda"))[0], ssd.ssd_draft_verify(*v)[0])
    with pytest.raises(ssd.SSDError):
        ssd.ssd_draft_verify(*v, workspace=torch.empty(n - 1, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("L,H,G,N", [(100, 4, 4, 64), (70, 6, 2, 128), (16000, 8, 2, 64), (33, 3, 3, 128)])
def test_workspaces_of_several_groups(ssd, dtype, L, H, G, N):
    """What the function says is enough for the groups it was told of, and not more than that."""
    a, o = inputs(1, L, H, G, 16, N, dtype)
    A, O = to(a), to(o)
    n = ssd.ssd_delta_workspace_size(1, L, H, 16, N, dtype, G)
    want = ssd.ssd_delta_fwd(**A, **O)
    space = torch.empty(n + 64, dtype=torch.uint8, device="cuda").fill_(0xA5)
    got = ssd.ssd_delta_fwd(**A, **O, workspace=space[:n])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bool((space[n:] == 0xA5).all())
    with pytest.raises(ssd.SSDError):
        ssd.ssd_delta_fwd(**A, **O, workspace=space[:n - 16])


def test_arguments_are_refused(ssd):
    a, o = inputs(2, 3, 4, 2, 64, 64, torch.bfloat16, cached=True)
    A, O = to(a), to(o)
    call = lambda **c: ssd.ssd_delta_fwd(**{**A, **O, **c})  # noqa: E731
    call()
    for change in (dict(x=A["x"].float()), dict(Bm=A["Bm"][:, :2]), dict(Cm=A["Cm"].transpose(2, 3).contiguous().transpose(2, 3)),
                   dict(beta=A["beta"].float()), dict(dt=A["dt"].cpu()), dict(A=A["A"][:3]), dict(A=None), dict(beta=None),
                   dict(norm_eps=-1.0), dict(norm_eps=float("nan")), dict(scale=float("inf")), dict(scale="x"), dict(slots=O["slots"].long()),
                   dict(init_state=O["init_state"][:3]), dict(final_state=None), dict(final_state=O["final_state"].bfloat16()),
                   dict(x=A["x"][..., :24].contiguous()), dict(y=torch.empty(2, 3, 4, 64, device="cuda")),
                   dict(lengths=torch.zeros(3, dtype=torch.int32, device="cuda")), dict(x=A["x"].half())):
        with pytest.raises(ssd.SSDError):
            call(**change)
    with pytest.raises(ssd.SSDError):  # rows for states that there are none of
        ssd.ssd_delta_fwd(**A, slots=O["slots"], want_final_state=False)
    v = dict(logits=torch.randn(2, 3, 50, device="cuda"), draft=torch.zeros(2, 2, dtype=torch.int32, device="cuda"),
             uniforms=torch.rand(2, 3, device="cuda"))
    for change in (dict(draft=v["draft"].long()), dict(draft=None), dict(uniforms=v["uniforms"][:, :2].contiguous()),
                   dict(draft_logits=v["logits"]), dict(draft_logits=v["logits"][:, :2].bfloat16()), dict(scale=torch.ones(3, device="cuda")),
                   dict(lengths=torch.ones(2, device="cuda")), dict(logits=v["logits"].transpose(1, 2)), dict(uniforms=None)):
        with pytest.raises(ssd.SSDError):
            ssd.ssd_draft_verify(**{**v, **change})


def test_offsets_past_32_bits(ssd):
    """Cache rows, tokens and logits that lie more than 2^31 values apart."""
    H, P, N = 2, 64, 128
    slots = torch.tensor([2 ** 31 // (H * P * N) + 3, 1], dtype=torch.int32)
    state = torch.empty(int(slots[0]) + 1, H, P, N, device="cuda")
    for L in (3, 40):
        a, o = inputs(2, L, H, 1, P, N, torch.bfloat16, seed=L)
        init = torch.randn(2, H, P, N) * 0.3
        state[slots.long().cuda()] = init.cuda()
        wide = torch.empty(2, 2 ** 30 + 2 ** 26, device="cuda", dtype=torch.bfloat16)  # batches, and tokens within one, far apart
        step = 2 ** 30 // L // 64 * 64
        x = wide[:, :step * L].view(2, L, step)[:, :, :H * P].unflatten(2, (H, P))
        x.copy_(a["x"])
        y, _ = ssd.ssd_delta_fwd(**{**to(a), "x": x}, **to(o), init_state=state, slots=slots.cuda(), final_state=state)
        ry, _, rf, _ = ref.delta(**a, **o, init_state=init)
        near("final", state[slots.long().cuda()], rf, 2.0 ** -18)
        near("y", y, ry, 2.0 ** -8)
    del state
    V = 1000
    g = torch.Generator().manual_seed(3)
    logits, near_ = torch.randn(2, 3, V, generator=g), torch.randn(2, 2, V, generator=g)
    wide = torch.empty(2 ** 32 + 2 ** 20, device="cuda", dtype=torch.bfloat16)
    far = wide.as_strided((2, 3, V), (2 ** 31 + 2 ** 18, 2 ** 30 // 2 + 8, 1))
    far.copy_(logits)
    q = wide.as_strided((2, 2, V), (2 ** 31 + 2 ** 18, 2 ** 30 // 2 + 8, 1), 5000)
    q.copy_(near_)
    args = dict(draft=torch.randint(0, V, (2, 2), generator=g).int(), uniforms=torch.rand(2, 3, generator=g))
    got = ssd.ssd_draft_verify(far, draft_logits=q, **to(args))
    want = ref.verify(logits.bfloat16(), draft_logits=near_.bfloat16(), **args)
    assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[1].cpu(), want[1])
