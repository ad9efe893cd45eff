"""The verification of drafted tokens at the ends of its ranges, against the same
loop in 64 bits as in test_gpu_verify (its docstring has the tolerances)."""
import pytest
import torch

from test_gpu_verify import run, ssd  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [2 ** 19, 2 ** 19 - 1])
def test_largest_vocabulary_of_equal_logits(ssd, V, dtype):  # noqa: F811
    """The sum of all weights is the largest there is (2^63 of their units for 2^19 equal logits).  The random
    numbers are odd multiples of 2^-24 (a token has 32 of 2^19), so that none falls on a token's border."""
    flat = torch.full((1, 1, V), 1.5, dtype=dtype)
    u = torch.tensor([0.0, 1 - 2.0 ** -24, 2.0 ** -24, 0.5 + 2.0 ** -24, 0.3 * 2 ** 24 // 2 * 2.0 ** -23 + 2.0 ** -24])
    got = run(ssd, dict(logits=flat.expand(5, 1, V), draft=torch.zeros(5, 0, dtype=torch.int32), uniforms=u[:, None]))
    assert got[0].flatten().tolist() == [int(v * V) for v in u.double()]
    # a draft's row of equal logits too: accepted, or outside the vocabulary, with nothing left of p - q
    draft = torch.tensor([[V - 1], [-1], [7]], dtype=torch.int32)
    uniforms = torch.stack([torch.tensor([0.75, 0.25, 0.0]), u[2:]], 1)
    got = run(ssd, dict(logits=flat.expand(3, 2, V), draft=draft, draft_logits=flat.expand(3, 1, V), uniforms=uniforms))
    assert got[1].tolist() == [1, 0, 1]
    # the draft's row flat, the target's not, and the other way round
    g = torch.Generator().manual_seed(V)
    steep = (torch.randn(1, 1, V, generator=g) * 2).to(dtype)
    draft[:, 0] = torch.tensor([int((steep < 0)[0, 0].long().argmax()), 5, 11])  # an unlikely one
    uniforms[:, 0] = 1 - 2.0 ** -24
    run(ssd, dict(logits=steep.expand(3, 2, V), draft=draft, draft_logits=flat.expand(3, 1, V), uniforms=uniforms))
    run(ssd, dict(logits=flat.expand(3, 2, V), draft=draft, draft_logits=steep.expand(3, 1, V), uniforms=uniforms))
    run(ssd, dict(logits=flat.expand(3, 2, V), draft=draft, uniforms=uniforms))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_drafts_that_hardly_have_a_weight(ssd, dtype):  # noqa: F811
    """Shares of e^-200 of a drafted token under both: their ratio decides, as for any other; 0 accepts what has any."""
    V = 300
    g = torch.Generator().manual_seed(9)
    target, near = torch.randn(V, generator=g).to(dtype), torch.randn(V, generator=g).to(dtype)
    for i, (p, q) in enumerate(((-200, -199), (-199, -200), (-150, -80), (-80, -150), (-120, -120.5))):
        target[10 * i], near[10 * i] = p, q
    target[60] = -float("inf")
    draft = torch.tensor([0, 0, 10, 20, 30, 40, 40, 20, 60, 0])
    u = torch.tensor([0.2, 0.6, 0.9, 0.0, 0.9, 0.5, 0.99, 0.5, 0.0, 0.0])
    a = dict(logits=target.expand(10, 2, V), draft=draft.int()[:, None], draft_logits=near.expand(10, 1, V),
             uniforms=torch.stack([u, torch.rand(10, generator=g)], 1))
    got = run(ssd, a)
    assert len(set(got[1].tolist())) == 2
    got = run(ssd, {**a, "draft_logits": None})
    assert got[1].tolist() == [0, 0, 0, 1, 0, 0, 0, 0, 0, 1]
    run(ssd, {**a, "scale": torch.full((10,), 3.0)})


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["noise", "one token", "two tokens exchanged", "a part"])
def test_drafts_almost_like_the_target(ssd, kind, dtype):  # noqa: F811
    """p and q are equal to 10^-5 or so, which 32-bit sums cannot tell for all tokens: what is drawn after a refusal is
    the 64-bit loop's.  (Weights are good to 2^-38 and p - q to 2^-38 10^5 of itself: no number is that near a
    token's border.)"""
    V, B = 3001, 48
    g = torch.Generator().manual_seed(5)
    target = torch.randn(V, generator=g).mul(2).to(dtype).float()
    near = target.clone()
    if kind == "noise":
        near = near + torch.randn(V, generator=g) * (1e-5 if dtype == torch.float32 else 0.0)
        if dtype == torch.bfloat16:  # (a last place, of a few tokens)
            i = torch.randperm(V, generator=g)[:9]
            near[i] = near[i] * (1 + 2.0 ** -7)
    elif kind == "one token":
        near[17] += 2.0 ** -7 * near[17].abs()
    elif kind == "two tokens exchanged":
        near[5], near[2900] = float(target[2900]), float(target[5])
    else:
        near[1500:] -= 1e-4 if dtype == torch.float32 else 2.0 ** -7 * near[1500:].abs()
    p, q = target.double().softmax(0), near.to(dtype).double().softmax(0)
    refused = int((p / q).argmin())
    assert float(p[refused] / q[refused]) < 1 - 2.0 ** -18
    u = torch.rand(B, 2, generator=g)
    u[:, 0] = 1 - 2.0 ** -24
    a = dict(logits=target.to(dtype).expand(B, 2, V), draft_logits=near.to(dtype).expand(B, 1, V),
             draft=torch.full((B, 1), refused, dtype=torch.int32), uniforms=u)
    rest = (p - q).clamp(min=0)
    border = (rest.cumsum(0) / rest.sum())[:, None] - u[:, 1].double()
    assert float(border.abs().min()) > 2.0 ** -38 / float(rest.sum()), "a number at a border"
    got = run(ssd, a)
    assert not got[1].any() and len(set(got[0][:, 0].tolist())) > (0 if kind == "two tokens exchanged" else 9)
