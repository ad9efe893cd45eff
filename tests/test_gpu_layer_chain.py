"""Calls that read what the call in front of them writes, again and again into
the same buffers: a launch is set up while the one in front still runs, and must
see what that one writes, not what lay there before."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
both_types = pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])


@pytest.fixture(scope="module")
def ssd():
    import mamba_ssd_forward_chunked_gb300 as m
    return m


def alternate(chain, inputs, rounds=40):
    """chain(input) for inputs in turn, with nothing in between, against each one waited for."""
    want = []
    for x in inputs:
        torch.cuda.synchronize()
        want.append([t.clone() for t in chain(x)])
        torch.cuda.synchronize()
    got = [[t.clone() for t in chain(inputs[i % len(inputs)])] for i in range(rounds)]
    torch.cuda.synchronize()
    for i, outs in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(outs, want[i % len(inputs)])), i


@both_types
@pytest.mark.parametrize("B,L,C,N", [(1, 200, 64, 16), (2, 70, 5120, 16), (1, 2000, 48, 16), (3, 1, 512, 16)],
                         ids=["few", "shared", "segments", "token"])
def test_scan_after_its_convolution(ssd, dtype, B, L, C, N):
    g = torch.Generator().manual_seed(L)
    rand = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    weight, A = rand(C + 2 * N, 4), -torch.rand(C, N, generator=g).cuda() * N
    out = [torch.empty(B, L, n, dtype=dtype, device="cuda") for n in (C, N, N)]
    y, h = torch.empty(B, L, C, dtype=dtype, device="cuda"), torch.empty(B, C, N, device="cuda")

    def chain(u):
        ssd.ssd_conv_fwd(u, weight, split=(C, N, N), out=out)
        x, Bm, Cm = out
        return ssd.ssd_selective_scan(x, x, A, Bm.unsqueeze(2), Cm.unsqueeze(2), z=x, delta_softplus=True, y=y, final_state=h)
    alternate(chain, [rand(B, L, C + 2 * N).to(dtype) for _ in range(2)])


@both_types
@pytest.mark.parametrize("M", [1, 8, 16])
@pytest.mark.parametrize("width", [512, 509], ids=["vectors", "odd"])
def test_products_after_each_other(ssd, dtype, M, width):
    g = torch.Generator().manual_seed(M)
    layers = []
    for _ in range(4):
        w = torch.randn(width, width, generator=g).cuda() / width ** 0.5
        layers.append(ssd.w4_quantize(w, 64))
    space = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    x, y = (torch.empty(M, width, dtype=dtype, device="cuda") for _ in range(2))

    def chain(first):
        ssd.ssd_w4_matvec(first, *layers[0], 64, y=x, workspace=space)
        ssd.ssd_w4_matvec(x, *layers[1], 64, y=y, workspace=space)
        ssd.ssd_w4_matvec(y, *layers[2], 64, y=x, workspace=space)
        ssd.ssd_w4_matvec(x, *layers[3], 64, y=y, add=x, workspace=space)
        return x, y
    alternate(chain, [torch.randn(M, width, generator=g).to(dtype).cuda() for _ in range(2)])


@both_types
@pytest.mark.parametrize("B,H,slots", [(1, 8, False), (24, 16, False), (24, 16, True)], ids=["one", "batch", "slots"])
def test_steps_in_place(ssd, dtype, B, H, slots):
    """Token after token on the same state and ring, which each launch finds as the one in front left them."""
    g = torch.Generator().manual_seed(B)
    rand = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    N = 128
    C = H * 64 + 2 * N
    A, D, weight = -torch.rand(H, generator=g).cuda(), rand(H), rand(C, 4) * 0.5
    state, ring = torch.empty(B, H, 64, N, device="cuda"), torch.empty(B, 4, C, dtype=dtype, device="cuda")
    rows = torch.arange(B, dtype=torch.int32, device="cuda") if slots else None
    positions = [torch.full((B,), t, dtype=torch.int32, device="cuda") for t in range(6)]
    y = [torch.empty(B, H, 64, dtype=dtype, device="cuda") for _ in range(6)]

    def chain(x):
        u, dt = x
        state.zero_()
        for t in range(6):
            ssd.ssd_step(u[t], dt[t], A, D, weight, None, state, ring, positions[t], dt_softplus=True, slots=rows, y=y[t])
        return [state, ring, *y]
    alternate(chain, [(rand(6, B, C).to(dtype), rand(6, B, H).to(dtype)) for _ in range(2)])
