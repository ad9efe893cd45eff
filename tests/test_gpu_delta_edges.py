"""The gated delta rule in chunks at values where it can go wrong, against the
recurrence in 64 bits (bounds: delta_ref)."""
import pytest
import torch

import delta_ref as ref
from layer_ref import check, store
from test_gpu_delta import inputs, near, run, ssd, to  # noqa: F401

pytestmark = pytest.mark.gpu

BOTH = pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])


def short(a):
    """Keys and queries of lengths near 1, for calls that take them as they are."""
    N = a["Bm"].shape[3]
    a["Bm"], a["Cm"] = a["Bm"] * N ** -0.5, a["Cm"] * N ** -0.5
    return a


@BOTH
@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("L", [65, 150])
@pytest.mark.parametrize("eps", [None, 1.0, 0.0, 1e-6])
def test_keys_of_zeros(ssd, L, N, eps, dtype):  # noqa: F811
    """All keys of a chunk are zero, or those of some tokens, the last among them: nothing is written then."""
    a, o = inputs(2, L, 4, 2, 32, N, dtype, cached=True, seed=L)
    short(a)
    a["Bm"][0, :64] = 0
    a["Bm"][1, 3::7] = 0
    a["Bm"][:, -1] = 0
    a["Cm"][:, 5:9] = 0
    run(ssd, a, {**o, "norm_eps": eps})
    a["Bm"][:] = 0
    y, final = run(ssd, a, {**o, "norm_eps": eps})
    o["lengths"] = torch.tensor([L - 1, 33], dtype=torch.int32)
    run(ssd, a, {**o, "norm_eps": eps})


def bounds(a, o):
    return ref.delta(**a, **o, spread=65.0, pt=2.0 ** (-12 if a["x"].dtype == torch.bfloat16 else -22))


@BOTH
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("H,P,N", [(2, 48, 128), (2, 32, 64), (80, 32, 64), (160, 16, 128)])  # every form of the walk
def test_values_that_are_not_finite_stay_in_their_channel(ssd, H, P, N, value, dtype):  # noqa: F811
    """One in x, in the second of four chunks, and one in a row of a state: the other channels are those of the
    recurrence without it, its own is not finite from there on and as it was before."""
    a, o = inputs(1, 200, H, H, P, N, dtype, seed=P)
    o["init_state"] = torch.randn(1, H, P, N, generator=torch.Generator().manual_seed(P)) * 0.3
    ry, by, rf, bf = bounds(a, o)
    by = store(ry, by, dtype)
    for where in ("x", "init_state"):
        bad = dict(a, **o)
        bad[where] = bad[where].clone()
        first = 64 if where == "x" else 0
        if where == "x":
            bad["x"][0, 100, 1, 5] = value
        else:
            bad["init_state"][0, 1, 5, 9] = value
        y, final = (v.cpu() for v in ssd.ssd_delta_fwd(**to(bad)))
        others = torch.ones(H, P, dtype=torch.bool)
        others[1, 5] = False
        check(where + ": y", y[:, :, others], ry[:, :, others], by[:, :, others])
        check(where + ": final", final[:, others], rf[:, others], bf[:, others])
        check(where + ": y before", y[:, :first, 1, 5], ry[:, :first, 1, 5], by[:, :first, 1, 5])
        assert not torch.isfinite(y[0, max(first, 101):, 1, 5]).any() and not torch.isfinite(final[0, 1, 5]).any()


@BOTH
@pytest.mark.parametrize("H,P,N", [(2, 48, 128), (80, 32, 64), (160, 16, 128)])
def test_bounds_past_32_bits(ssd, H, P, N, dtype):  # noqa: F811
    """Values so large that 64 times them is no number: a channel of them keeps its digits, and so does a state."""
    a, o = inputs(1, 200, H, H, P, N, dtype, seed=P)
    a["x"][0, :, 1, 5] = a["x"][0, :, 1, 5] * 2.0 ** 123
    o["init_state"] = torch.randn(1, H, P, N, generator=torch.Generator().manual_seed(P))
    o["init_state"][0, 0, 3] *= 2.0 ** 124
    y, final = ssd.ssd_delta_fwd(**to(a), **to(o))
    ry, _, rf, _ = ref.delta(**a, **o)
    for h, p in ((1, 5), (0, 3)):
        near("final", final[0, h, p], rf[0, h, p], 2.0 ** -19)
        near("y", y[0, :, h, p], ry[0, :, h, p], 2.0 ** -19 if dtype == torch.float32 else 2.0 ** -8)
    assert torch.isfinite(y).all() and torch.isfinite(final).all()


@pytest.mark.parametrize("B,L,H,G,P,N", [(1, 25000, 16, 16, 64, 64), (4, 4096, 32, 16, 128, 128)])
def test_repeated_calls_give_the_same(ssd, B, L, H, G, P, N):  # noqa: F811
    """Factors that a warp had not read yet were replaced by those of two chunks later, in one call of some 400."""
    a, o = inputs(B, L, H, G, P, N, torch.bfloat16, seed=1)
    A, O = to(a), to(o)
    y, final = ssd.ssd_delta_fwd(**A, **O)
    other = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(2500):
        y2, final2 = ssd.ssd_delta_fwd(**A, **O)
        other += (y2 != y).any().long() + (final2 != final).any().long()
    assert int(other) == 0 and torch.isfinite(y.float()).all() and torch.isfinite(final).all()

@BOTH
@pytest.mark.parametrize("eps", [None, 1e-6])
def test_the_last_key_alone_and_forgotten_ones(ssd, eps, dtype):  # noqa: F811
    """A chunk whose only token with a key is its first, forgotten by 2^-100 and more at its end."""
    a, o = inputs(1, 128, 3, 1, 48, 128, dtype, seed=4)
    short(a)
    a["Bm"][0, 1:64] = 0
    for gate in (1.0, 5.0, 50.0):  # times 63 tokens
        a["dt"] = torch.full_like(a["dt"], gate)
        a["A"] = torch.tensor([-0.5, -1.0, -3.0])
        run(ssd, a, dict(beta_sigmoid=True, norm_eps=eps))


@BOTH
@pytest.mark.parametrize("L,N", [(90, 64), (90, 128), (200, 64), (200, 128)])
def test_plain_arguments(ssd, L, N, dtype):  # noqa: F811
    """No norms, no activations, a scale of its own, 32-bit gates beside bf16."""
    a, o = inputs(2, L, 2, 2, 64, N, dtype, gates=torch.float32, seed=9)
    a["Bm"], a["Cm"] = a["Bm"] * N ** -0.5, a["Cm"] * 0.5
    a["dt"], a["beta"] = a["dt"].abs() * 0.1, torch.rand(2, L, 2, generator=torch.Generator().manual_seed(L)) * 2
    run(ssd, a, dict(scale=-0.75))


@BOTH
@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("length", [1e-17, 1e-7, 1e-3, 1.0, 30.0, 1000.0, 1e17, "mixed"])
def test_keys_of_any_length(ssd, length, N, dtype):  # noqa: F811
    """Keys as they are, beta |k|^2 between 0.3 and 1: the same digits whatever their length, also where every token
    has another.  (Over all values as in test_prompts.)"""
    g = torch.Generator().manual_seed(N)
    a, _ = inputs(2, 150, 4, 2, 48, N, dtype, gates=torch.float32, seed=5)
    size = torch.full((2, 150, 2, 1), length) if length != "mixed" else 10.0 ** (torch.rand(2, 150, 2, 1, generator=g) * 6 - 3)
    a["Bm"] = (a["Bm"].float() / a["Bm"].float().norm(dim=-1, keepdim=True) * size).to(dtype)
    a["Cm"] = (a["Cm"].float() * 10.0 ** (torch.rand(2, 150, 2, 1, generator=g) * 20 - 10)).to(dtype)
    a["dt"] = a["dt"].abs() * 0.1
    share = 0.3 + 0.7 * torch.rand(2, 150, 4, generator=g)
    a["beta"] = (share.double() / size.double().square().repeat_interleave(2, 2)[..., 0]).float()
    o = dict(init_state=torch.randn(2, 4, 48, N, generator=g) / size[:, :1, :1, :, None].mean())
    y, final = run(ssd, a, o)
    ry, _, rf, _ = ref.delta(**a, **o)
    near("final", final, rf, 2.0 ** -19)
    near("y", y, ry, 2.0 ** -19 if dtype == torch.float32 else 2.0 ** -8)


@BOTH
@pytest.mark.parametrize("L,N", [(100, 64), (180, 128)])
def test_rules_that_grow(ssd, L, N, dtype):  # noqa: F811
    """One key for all tokens and beta |k|^2 = 2.25: a value becomes -1.25 times itself a token, 10^6 times a chunk.
    What a product loses grows as the values do, so it stays 2^-22 of them: 2^-17 for all of a state's chunks."""
    a, o = inputs(1, L, 2, 1, 32, N, dtype, gates=torch.float32, seed=6)
    a["Bm"] = torch.full((1, L, 1, N), (1.0 / N) ** 0.5 if N == 64 else 0.125 * 0.5).to(dtype)  # (exact; |k|^2 is 1, or 0.5)
    a["dt"][:] = 0.0
    a["beta"][:] = 2.25 if N == 64 else 4.5
    y, final = run(ssd, a, {})
    ry, _, rf, _ = ref.delta(**a)
    near("final", final, rf, 2.0 ** -17)
    near("y", y, ry, 2.0 ** -17 if dtype == torch.float32 else 2.0 ** -8)


@BOTH
@pytest.mark.parametrize("L,N", [(9, 64), (9, 256), (70, 64), (70, 128)])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_norms_of_rows_whose_squares_leave_32_bits(ssd, L, N, eps, dtype):  # noqa: F811
    """Rows of 10^-30 to 10^30, a single small value, and zeros.  In chunks the values to be written, r, of 64 tokens have
    one power of two: their second parts end at 2^-25 of a unit, and the bound that sets it, max |x| + sqrt(N) max |h|
    at most (beta and decays are below 1), is below 2^15 units and above 2^14, so each is off by 2^-39 of that bound
    whatever its own size.  A token's y has 64 of them at most, times |scale q| and a key of length below 1.42."""
    a, o = inputs(1, L, 2, 2, 32, N, dtype, seed=N)
    g = torch.Generator().manual_seed(L)
    for k in ("Bm", "Cm"):
        a[k] = (a[k].float() * 10.0 ** torch.randint(-30, 31, (1, L, 2, 1), generator=g)).to(dtype)
        a[k][0, 4] = 0
        a[k][0, 5, 0] = 0
        a[k][0, 5, 0, 7] = 1e-35
    o["norm_eps"] = eps
    y, final = ssd.ssd_delta_fwd(**to(a), **to(o))
    ry, by, rf, bf = ref.delta(**a, **o, spread=65.0 if L >= 32 else 1.0, pt=2.0 ** (-12 if dtype == torch.bfloat16 else -22))
    if L >= 32:
        h = 0.0
        for t in range(L + 1):
            h = max(h, float(ref.delta(**{k: v[:, :t] if v.dim() > 1 else v for k, v in a.items()}, **o)[2].abs().max()))
        floor = 2.0 ** -39 * 64 * 1.42 * (float(a["x"].abs().max()) + N ** 0.5 * h)
        q = a["Cm"].double()
        size = q.square().sum(-1) + eps
        length = torch.where(size > 0, q.norm(dim=-1) * size.rsqrt(), 0.0)
        by += floor * N ** -0.5 * length[..., None]
        bf += floor
    check("y", y, ry, store(ry, by, dtype))
    check("final", final, rf, bf)


@BOTH
@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("of", ["channels", "tokens", "heads"])
def test_values_of_different_sizes(ssd, of, N, dtype):  # noqa: F811
    """x of sizes from 1 to 10^4 by channel, by token (every 13th large) or by head, the smallest ones' digits.  The
    large ones set the powers of two of a block's columns: with X their largest, the bound of the state is up to
    64 1.42 (1 + sqrt(N)) X = 2^11 X, and its second parts end at 2^-39 of that, 2^-28 X, or 2^-13 for X = 4 10^4 beside
    values of 1: 2^-12 of the small channels' states over all values.  A head has bounds of its own: 2^-19."""
    a, o = inputs(1, 260, 4, 4, 32, N, torch.float32, seed=8)
    size = torch.ones(1, 260, 4, 32)
    if of == "channels":
        size *= 10.0 ** torch.arange(32).remainder(5)
    elif of == "tokens":
        size[:, ::13] *= 1e4
    else:
        size[:, :, 1::2] *= 1e4
    a["x"] = (a["x"] * size).to(dtype)
    for k in ("Bm", "Cm", "dt", "beta"):
        a[k] = a[k].to(dtype)
    y, final = run(ssd, a, o)
    ry, _, rf, _ = ref.delta(**a, **o)
    small = {"channels": (slice(None), slice(0, 32, 5)), "tokens": (slice(None), slice(None)), "heads": (slice(0, 4, 2), slice(None))}[of]
    loss = 2.0 ** -12 if of == "channels" else 2.0 ** -19
    near("final", final[:, small[0], small[1]], rf[:, small[0], small[1]], loss)
    near("y", y[:, :, small[0], small[1]], ry[:, :, small[0], small[1]], loss if dtype == torch.float32 else 2.0 ** -8)
