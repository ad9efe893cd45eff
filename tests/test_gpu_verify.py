"""The verification of drafted tokens against a loop over them in 64 bits.

Tokens and counts have to be those of the reference.  A random number within
2^-20 of an acceptance's border, or within 2^-34 of a token's, may fall either
way (32-bit sums; weights to 2^-38 over a vocabulary's sums): the inputs here are
fixed, and none is that near.  Log-probabilities: the difference of a logit from
the maximum and the sum's logarithm, 2^-20 of each and of 1."""
import pytest
import torch

import delta_ref as ref

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module")
def ssd():
    import mamba_ssd_forward_chunked_gb300 as m
    return m


def inputs(B, T, V, dtype=torch.float32, probs=True, seed=0):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(B, T + 1, V, generator=g) * 3
    near = logits[:, :T] + torch.randn(B, T, V, generator=g) * 0.7
    draft = (near - torch.log(-torch.log(torch.rand(B, T, V, generator=g).clamp(1e-7, 1 - 1e-7)))).argmax(-1) if T else torch.zeros(B, 0)
    return dict(logits=logits.to(dtype), draft=draft.to(torch.int32), uniforms=torch.rand(B, T + 1, generator=g),
                draft_logits=near.to(dtype) if probs else None)


def to(a):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in a.items()}


def run(ssd, a):
    got = [v.cpu() for v in ssd.ssd_draft_verify(**to(a))]
    want = ref.verify(**a)
    assert torch.equal(got[1], want[1]), (got[1], want[1])
    assert torch.equal(got[0], want[0]), (got[0], want[0])
    scale = torch.ones(got[2].shape[0]) if a.get("scale") is None else a["scale"]
    size = a["logits"].double().masked_fill(~torch.isfinite(a["logits"].double()), 0).abs().amax((1, 2)) * scale.double()
    bound = 2.0 ** -20 * (1 + want[2].abs() + 2 * size.masked_fill(~torch.isfinite(size), 0)[:, None])
    assert ((got[2].double() - want[2]).abs() <= bound)[want[0] >= 0].all() and not got[2][want[0] < 0].any()
    return got


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("B,T,V", [(1, 1, 1), (2, 0, 9), (3, 2, 7), (5, 4, 255), (2, 8, 257), (7, 3, 1000), (2, 5, 4097),
                                   (3, 4, 32768), (1, 64, 513), (2, 2, 131072), (1, 1, 262147)])
def test_sizes(ssd, B, T, V, probs, dtype):
    for seed in range(3):
        a = inputs(B, T, V, dtype, probs, seed)
        if not probs:  # drafts that are likely
            a["draft"] = a["logits"][:, :T].float().argmax(-1).to(torch.int32)
        run(ssd, a)


def test_many_requests(ssd):
    got = run(ssd, inputs(200, 5, 301, torch.bfloat16))
    assert len(set(got[1].tolist())) == 6  # every count occurs


def test_scale_and_lengths(ssd):
    a = inputs(9, 4, 1003, seed=2)
    a["scale"] = torch.tensor([1.0, 0.5, 2.0, 1e-3, 30.0, 0.0, -1.0, INF, float("nan")])
    a["lengths"] = torch.tensor([4, 0, 2, -5, 9, 4, 4, 4, 4], dtype=torch.int32)
    got = run(ssd, a)
    assert (got[0][5:] == -1).all() and not got[1][5:].any()


def test_strides_and_alignment(ssd):
    for dtype in (torch.float32, torch.bfloat16):
        a = inputs(3, 3, 1000, dtype, seed=3)
        want = ssd.ssd_draft_verify(**to(a))
        for pad in (1, 3, 8):
            wide = torch.full((3, 7, 1000 + pad), INF, dtype=dtype)
            wide[:, :4, pad:], wide[:, 4:, pad:] = a["logits"], a["draft_logits"]
            dev = wide.cuda()
            got = ssd.ssd_draft_verify(dev[:, :4, pad:], a["draft"].cuda(), a["uniforms"].cuda(), draft_logits=dev[:, 4:, pad:])
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_random_numbers_at_the_ends(ssd):
    """0 draws the first token with any weight, the largest number below 1 the last."""
    a = inputs(4, 1, 700, seed=4)
    a["logits"][:, :, :5] = -INF
    a["logits"][:, :, -3:] = -INF
    a["uniforms"] = torch.tensor([[0.0, 0.0], [0.0, 1 - 2.0 ** -24], [1 - 2.0 ** -24, 0.0], [0.5, 1 - 2.0 ** -24]])
    run(ssd, a)
    b = inputs(1, 0, 700, seed=5)
    b["logits"][:, :, :5] = -INF
    for u, v in ((0.0, 5), (-1.0, 5), (float("nan"), 5)):
        b["uniforms"] = torch.tensor([[u]])
        assert int(ssd.ssd_draft_verify(**to(b))[0]) == v
    for u in (1.0, 2.0, INF):
        b["uniforms"] = torch.tensor([[u]])
        assert int(ssd.ssd_draft_verify(**to(b))[0]) == 699


def test_equal_distributions(ssd):
    """p = q: everything is accepted, whatever the numbers."""
    a = inputs(6, 4, 333, seed=6)
    a["logits"][:, :4] = a["draft_logits"]
    got = run(ssd, a)
    assert (got[1] == 4).all()


def test_masked_and_odd_logits(ssd):
    a = inputs(8, 2, 130, seed=7)
    a["logits"][0, 0] = -INF                      # the target allows nothing
    a["logits"][1] = torch.finfo(torch.float32).min   # the type's lowest value everywhere
    a["draft_logits"][2] = -INF                   # a draft without a distribution
    a["logits"][3, :, 5:] = -INF
    a["logits"][4, 0, 7] = INF
    a["logits"][4, 0, 9] = INF
    a["logits"][5, 0, 3] = float("nan")
    a["draft_logits"][5, 0, 8] = float("nan")
    a["draft"][6] = torch.tensor([-1, 5])
    a["draft"][7] = torch.tensor([130, 5])
    run(ssd, a)
    a["draft_logits"] = None
    run(ssd, a)


def test_nothing_left_of_the_difference(ssd):
    """A rejected draft (it has no weight under either) where p = q: p itself is drawn from."""
    a = inputs(2, 1, 50, seed=8)
    a["logits"][:, 0] = a["draft_logits"][:, 0]
    a["logits"][:, 0, 4] = a["draft_logits"][:, 0, 4] = -INF
    a["draft"][:] = 4
    got = run(ssd, a)
    assert not got[1].any()


@pytest.mark.parametrize("V", [50001, 131072])
@pytest.mark.parametrize("width", [1.0, 3.0, 6.0])
def test_drawn_tokens_are_those_of_64_bits(ssd, V, width):
    """Many numbers over flat and over steep distributions, where most tokens have less than 1e-5 of them."""
    g = torch.Generator().manual_seed(11)
    logits = (width * torch.randn(1, 1, V, generator=g)).expand(2048, 1, V)
    u = torch.rand(2048, 1, generator=g)
    got = ssd.ssd_draft_verify(logits.cuda(), torch.zeros(2048, 0, dtype=torch.int32).cuda(), u.cuda())[0].cpu()
    c = torch.softmax(logits[0, 0].double(), 0).cumsum(0)
    assert torch.equal(got[:, 0].long(), torch.searchsorted(c, u[:, 0].double() * c[-1], right=True))
