"""Values and arguments of the layer operators that the wider tests' bounds are
too wide, or too few, to see."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ssd():
    import mamba_ssd_forward_chunked_gb300 as m
    return m


@pytest.mark.parametrize("how", ["step", "token", "prompt"])
def test_softplus_has_no_bias(ssd, how):
    """Steps are added up over a whole prompt, so their softplus must not lean to
    one side: half a unit of a 32-bit number in [1/2, 1), 3e-8, which is 4.3e-8 of
    log 2, and a tenth more."""
    C = 4096
    v = torch.linspace(-0.05, 0.05, C)
    one = torch.ones(1, 1, C, device="cuda")
    if how == "step":  # y = softplus(dt) x.b c: x = b = c = 1, one state of 64 counts
        H, N = C, 64
        channels = H * 64 + 2 * N
        u = torch.zeros(1, channels, device="cuda")
        u[:, :H * 64], u[:, H * 64], u[:, H * 64 + N] = 1.0, 1.0, 1.0
        weight = torch.zeros(channels, 2, device="cuda")
        state, ring = torch.zeros(1, H, 64, N, device="cuda"), torch.zeros(1, 2, channels, device="cuda")
        weight[:, 1] = 20.0  # silu(20) = 20 - 4e-8
        ssd.ssd_step(u, v.view(1, C).cuda(), torch.zeros(H, device="cuda"), torch.zeros(H, device="cuda"), weight, None,
                     state, ring, torch.zeros(1, dtype=torch.int32, device="cuda"), dt_softplus=True)
        got = state[0, :, 0, 0].double().cpu() / 400.0
    else:  # the state is the last step's d u b: in the prompt nothing is left of the first
        L = 1 if how == "token" else 2
        x, b = one.expand(1, L, C).contiguous(), torch.ones(1, L, 1, 1, device="cuda")
        delta = v.cuda().view(1, 1, C).expand(1, L, C).contiguous()
        _, h = ssd.ssd_selective_scan(x, delta, torch.full((C, 1), -1000.0, device="cuda"), b, b, delta_softplus=True)
        got = h[0, :, 0].double().cpu()
    want = torch.log1p(torch.exp(v.double()))
    assert abs(float(((got - want) / want).mean())) < 4.7e-8


def test_flags_that_are_neither(ssd):
    """What has no truth value is an error of its own, not a lost one."""
    z = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    two = z(2)
    step = (z(2, 384), z(2, 4), z(4), z(4), z(384, 4), None, z(2, 4, 64, 64), z(2, 4, 384), z(2).to(torch.int32))
    with pytest.raises(RuntimeError, match="ambiguous"):
        ssd.ssd_step(*step, dt_softplus=two)
    scan = (z(2, 1, 12), z(2, 1, 12), z(12, 16), z(2, 1, 1, 16), z(2, 1, 1, 16))
    for flag in ("delta_softplus", "want_final_state"):
        with pytest.raises(RuntimeError, match="ambiguous"):
            ssd.ssd_selective_scan(*scan, **{flag: two})


def test_conv_ring_of_more_channels_than_32_bit_offsets_reach(ssd):
    """The last of a ring's slots begins beyond 2^31 elements of its row."""
    C, W = 720_000_016, 4
    ring = torch.zeros(1, W, C, dtype=torch.bfloat16, device="cuda")
    for q in range(W):
        ring[0, q, ::4096], ring[0, q, -1] = 1.0 + q, 5.0 + q
    new = torch.full_like(ring, 9.0)
    ssd.ssd_conv_fwd(torch.empty(1, 0, C, dtype=torch.bfloat16, device="cuda"), torch.zeros(C, W, device="cuda"),
                     ring=ring, new_ring=new)
    assert torch.equal(ring, new)
