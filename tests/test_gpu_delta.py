"""The gated delta rule against its recurrence in 64 bits."""
import pytest
import torch

import delta_ref as ref
from layer_ref import check, store

pytestmark = pytest.mark.gpu

NORM = 1e-6


@pytest.fixture(scope="module")
def ssd():
    import mamba_ssd_forward_chunked_gb300 as m
    return m


def inputs(B, L, H, G, P, N, dtype=torch.float32, cached=False, seed=0, gates=None):
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    gates = gates or dtype
    a = dict(x=rand(B, L, H, P).to(dtype), dt=(rand(B, L, H) * 0.5).to(gates), A=-torch.exp(torch.rand(H, generator=g) * 2.7),
             Bm=rand(B, L, G, N).to(dtype), Cm=rand(B, L, G, N).to(dtype), beta=rand(B, L, H).to(gates))
    o = dict(dt_bias=torch.linspace(-5.0, -2.0, H), dt_softplus=True, beta_sigmoid=True, norm_eps=NORM)
    if cached:
        S = B + 2
        o["init_state"] = rand(S, H, P, N) * 0.3
        o["slots"] = torch.randperm(S, generator=g)[:B].to(torch.int32)
        o["final_state"] = torch.full((S, H, P, N), 7.0)
    return a, o


def to(d, dev="cuda"):
    return {k: v.to(dev) if isinstance(v, torch.Tensor) else v for k, v in d.items()}


def run(ssd, a, o, **more):
    spread = 65.0 if a["x"].shape[1] >= 32 and a["Bm"].shape[3] < 256 else 1.0  # in chunks, or token by token
    y, final = ssd.ssd_delta_fwd(**to(a), **to({**o, **more}))
    torch.cuda.synchronize()
    ry, by, rf, bf = ref.delta(**a, **{k: v for k, v in {**o, **more}.items() if k not in ("want_final_state", "y")}, spread=spread,
                               pt=2.0 ** (-12 if a["x"].dtype == torch.bfloat16 else -22))
    check("y", y, ry, store(ry, by, a["x"].dtype))
    if final is not None:
        check("final", final, rf, bf)
    return y, final


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,L,H,G,P,N", [
    (1, 1, 1, 1, 128, 128), (2, 1, 3, 1, 64, 64), (3, 5, 4, 2, 128, 128), (2, 16, 2, 2, 16, 128), (1, 17, 6, 3, 48, 64),
    (2, 33, 4, 1, 80, 256), (1, 31, 2, 1, 272, 128), (5, 2, 2, 2, 128, 256), (1, 1, 2, 1, 1024, 64)])
def test_tokens(ssd, B, L, H, G, P, N, dtype):
    a, o = inputs(B, L, H, G, P, N, dtype, seed=L + P)
    run(ssd, a, o)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("L", [1, 4, 19, 40])
def test_cache_rows_lengths_and_positions(ssd, L, dtype):
    a, o = inputs(5, L, 4, 2, 128, 128, dtype, cached=True, seed=3)
    o["lengths"] = torch.tensor([L, 0, L - 1, -3, L + 9], dtype=torch.int32)
    o["positions"] = torch.tensor([4, 2, 0, 0, 1], dtype=torch.int32)
    run(ssd, a, o)
    o["slots"][0], o["slots"][4] = 7, -1  # idle
    y, final = run(ssd, a, o)
    assert not y[0].any() and not y[4].any()


def near(name, got, want, bound):
    err = float((got.double().cpu() - want).norm() / want.norm())
    assert err <= bound, (name, err)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,L,H,G,P,N", [
    (1, 32, 2, 1, 64, 128), (1, 47, 2, 2, 16, 64), (1, 64, 1, 1, 64, 64), (1, 64, 2, 1, 128, 128), (2, 65, 2, 2, 32, 128), (1, 127, 4, 2, 16, 64), (2, 128, 3, 1, 48, 128),
    (1, 129, 2, 2, 80, 64), (1, 321, 6, 3, 128, 128), (3, 200, 2, 1, 144, 128), (40, 70, 4, 4, 64, 64), (20, 64, 8, 4, 48, 128)])
def test_prompts(ssd, B, L, H, G, P, N, dtype):
    """Whole prompts.  Over all rows the roundings are independent: 2^-19 of the state (three products a chunk, a
    few 2^-22 each), of y as well, and y is rounded once more."""
    a, o = inputs(B, L, H, G, P, N, dtype, seed=L + P)
    y, final = run(ssd, a, o)
    ry, _, rf, _ = ref.delta(**a, **o)
    near("final", final, rf, 2.0 ** -19)
    near("y", y, ry, 2.0 ** -19 if dtype == torch.float32 else 2.0 ** -8)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("L,N", [(64, 128), (150, 64), (257, 128)])
def test_prompts_in_a_cache(ssd, L, N, dtype):
    a, o = inputs(6, L, 4, 2, 64, N, dtype, cached=True, seed=3)
    o["lengths"] = torch.tensor([L, 0, L - 1, 63, L + 9, 1], dtype=torch.int32)
    o["positions"] = torch.tensor([4, 2, 0, 0, 1, 7], dtype=torch.int32)
    y, final = run(ssd, a, o)
    o["slots"][0], o["slots"][4] = 9, -1  # idle
    y2, _ = run(ssd, a, o)
    assert not y2[0].any() and not y2[4].any() and torch.equal(y[[1, 2, 3, 5]], y2[[1, 2, 3, 5]])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_prompt_is_its_tokens(ssd, dtype):
    """A prompt, and the same one resumed in pieces and token by token."""
    a, o = inputs(2, 200, 4, 2, 128, 128, dtype, seed=12)
    y, final = ssd.ssd_delta_fwd(**to(a), **to(o))
    state, ys = None, []
    for lo, hi in ((0, 100), (100, 170), (170, 171), (171, 180), (180, 200)):
        part = {k: v[:, lo:hi] if v.dim() > 1 else v for k, v in to(a).items()}
        yp, state = ssd.ssd_delta_fwd(**part, **to(o), init_state=state)
        ys.append(yp)
    near("final", state, final.double().cpu(), 2.0 ** -18)
    near("y", torch.cat(ys, 1), y.double().cpu(), 2.0 ** (-18 if dtype == torch.float32 else -7))


def test_many_chunks_in_pairs_of_launches(ssd):
    """So many heads and chunks that a call makes several pairs of launches, which overlap (also when replayed)."""
    for H, L in ((16, 4500), (16, 25000), (160, 3400)):
        a, o = inputs(1, L, H, H, 64, 64, torch.bfloat16, seed=H)
        A, O = to(a), to(o)
        y, final = ssd.ssd_delta_fwd(**A, **O)
        state, ys = None, []
        for lo in range(0, L, 640):
            part = {k: v[:, lo:lo + 640] if v.dim() > 1 else v for k, v in A.items()}
            yp, state = ssd.ssd_delta_fwd(**part, **O, init_state=state)
            ys.append(yp)
        near("final", state, final.double().cpu(), 2.0 ** -18)
        near("y", torch.cat(ys, 1), y.double().cpu(), 2.0 ** -7)
        for _ in range(20):
            y2, final2 = ssd.ssd_delta_fwd(**A, **O)
            assert torch.equal(y, y2) and torch.equal(final, final2)
        side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=side):
            y3, final3 = ssd.ssd_delta_fwd(**A, **O)
        for _ in range(10):
            y3.fill_(float("nan"))
            graph.replay()
            assert torch.equal(y, y3) and torch.equal(final, final3)


def test_strong_and_weak_decay(ssd):
    for shift in (-8.0, 4.0):
        a, o = inputs(1, 300, 2, 1, 64, 128, torch.bfloat16, seed=13)
        o["dt_bias"] = torch.full((2,), shift)
        run(ssd, a, o)
    a["A"] = a["A"].abs() * 0.1  # (growth)
    o["dt_bias"] = torch.full((2,), -3.0)
    run(ssd, a, o)
    a["A"], o["dt_bias"] = -a["A"] * 10, torch.full((2,), 4.0)
    a["dt"][0, 50:60] = 300.0  # forgets everything, several times
    a["dt"][0, 130] = 300.0
    run(ssd, a, o)


def test_rows_of_nobody_stay(ssd):
    a, o = inputs(2, 3, 2, 1, 64, 64, cached=True)
    o["slots"] = torch.tensor([3, 1], dtype=torch.int32)
    _, final = run(ssd, a, o)
    assert (final[[0, 2]] == 7.0).all()


def test_in_place_and_without_a_state(ssd):
    a, o = inputs(3, 9, 4, 2, 128, 128, torch.bfloat16, cached=True, seed=5)
    y, final = run(ssd, a, o)
    state = o["init_state"].cuda()
    y2, same = ssd.ssd_delta_fwd(**to(a), **to({**o, "init_state": state, "final_state": state}))
    assert same.data_ptr() == state.data_ptr() and torch.equal(y, y2)
    rows = o["slots"].long().cuda()
    assert torch.equal(state[rows], final[rows])
    others = [i for i in range(5) if i not in o["slots"].tolist()]
    assert torch.equal(state[others].cpu(), o["init_state"][others])
    y3, none = ssd.ssd_delta_fwd(**to(a), **to({**o, "final_state": None, "want_final_state": False}))
    assert none is None and torch.equal(y, y3)


def test_plain_arguments(ssd):
    """No norms, no activations, a scale of its own, 32-bit gates beside bf16."""
    a, o = inputs(2, 11, 2, 2, 64, 64, torch.bfloat16, gates=torch.float32, seed=9)
    a["Bm"], a["Cm"] = a["Bm"] * 0.125, a["Cm"] * 0.5
    a["dt"], a["beta"] = a["dt"].abs() * 0.1, torch.rand(2, 11, 2) * 2
    run(ssd, a, dict(scale=-0.75))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("L", [21, 90])
def test_strides(ssd, L, dtype):
    B, H, G, P, N = 2, 4, 2, 64, 128
    a, o = inputs(B, L, H, G, P, N, dtype, seed=2)
    for pad in (0, 8, 3):  # 16-byte rows and others
        wide = torch.zeros(B, L, H * P + 2 * G * N + 2 * H + pad, dtype=dtype)
        parts = [H * P, G * N, G * N, H, H]
        views = [v.unflatten(2, s) if s else v for v, s in zip(wide[:, :, pad:].split(parts, 2), [(H, P), (G, N), (G, N), None, None])]
        for v, k in zip(views, ("x", "Bm", "Cm", "dt", "beta")):
            v.copy_(a[k])
        dev = wide.cuda()
        views = [v.unflatten(2, s) if s else v for v, s in zip(dev[:, :, pad:].split(parts, 2), [(H, P), (G, N), (G, N), None, None])]
        y, final = ssd.ssd_delta_fwd(views[0], views[3], a["A"].cuda(), views[1], views[2], views[4], **to(o))
        want, wantf = ssd.ssd_delta_fwd(**to(a), **to(o))
        assert torch.equal(y, want) and torch.equal(final, wantf)
    t = a["x"].transpose(0, 1).contiguous().cuda().transpose(0, 1)  # the batch inside
    y2, _ = ssd.ssd_delta_fwd(**to({**a, "x": t}), **to(o))
    assert torch.equal(want, y2)


def test_values_at_the_edge(ssd):
    """Zero rows with and without an epsilon, a gate that forgets everything, beta 0 and 1."""
    a, o = inputs(1, 6, 2, 1, 64, 64, seed=4)
    a["Bm"][0, 1] = 0
    a["Cm"][0, 2] = 0
    a["dt"][0, 3] = 200.0
    a["beta"][0, 4] = -200.0
    a["beta"][0, 5] = 200.0
    run(ssd, a, o)
    run(ssd, a, {**o, "norm_eps": 0.0})


@pytest.mark.parametrize("L,N", [(40, 128), (150, 64), (150, 128)])
def test_masked_tokens_may_hold_anything(ssd, L, N):
    a, o = inputs(2, L, 2, 1, 128, N, torch.bfloat16, cached=True, seed=6)
    o["lengths"] = torch.tensor([L - 17, 7], dtype=torch.int32)
    y, final = ssd.ssd_delta_fwd(**to(a), **to(o))
    for b, n in enumerate((L - 17, 7)):
        for k in ("x", "Bm", "Cm", "dt", "beta"):
            a[k][b, n:] = float("nan")
    y2, final2 = ssd.ssd_delta_fwd(**to(a), **to({**o, "final_state": o["final_state"].clone()}))
    assert torch.equal(y, y2) and torch.equal(final, final2)


def test_empty(ssd):
    a, o = inputs(2, 0, 2, 1, 64, 64, cached=True)
    y, final = ssd.ssd_delta_fwd(**to(a), **to(o))
    rows = o["slots"].long()
    assert y.shape == (2, 0, 2, 64) and torch.equal(final.cpu()[rows], o["init_state"][rows])
    a, o = inputs(0, 3, 2, 1, 64, 64)
    assert ssd.ssd_delta_fwd(**to(a), **to(o))[0].shape == (0, 3, 2, 64)
