"""examples/beam_search.py: prompts, single tokens, 4-bit projections, selection
and the reordering of states together."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("beam_search_example", os.path.join(ROOT, "examples", "beam_search.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


# What a sequence's score may differ by between the token-by-token path and the prompt path over
# the same tokens: the prompt's products are TF32 (2^-11 each factor) or bf16 (2^-9 on every value
# that is stored between operators); some 20 such roundings a layer and token act on logits of size 1 to 4.
TOL = {torch.float32: 0.02, torch.bfloat16: 0.15}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("L", [1, 2, 70])
def test_scores_are_those_of_the_sequences(ex, dtype, L):
    """Every hypothesis' score is the log-probability that the prompt path gives
    its tokens: a state that followed the wrong beam would be off by whole units."""
    model = ex.Model(vocab=300, width=128, layers=2, dtype=dtype, seed=3)
    g = torch.Generator().manual_seed(L)
    B, W, T = 3, 4, 9
    prompt = torch.randint(0, 300, (B, L), generator=g).cuda()
    tokens, scores = ex.beam_search(model, prompt, W, T, eos=299)
    assert tokens.shape == (B, W, T) and (scores[:, :-1] >= scores[:, 1:]).all()
    whole = torch.cat([prompt[:, None].expand(B, W, L), tokens.long()], 2).reshape(B * W, L + T)
    logits, _ = model.prompt(whole)
    logp = torch.log_softmax(logits.float(), -1)[:, L - 1:-1]
    each = logp.gather(2, whole[:, L:, None])[..., 0].view(B, W, T)
    after = (torch.cumsum((tokens == 299).int(), -1) - (tokens == 299).int()) > 0  # after the end: free
    want = torch.where(after, 0.0, each).sum(-1)
    assert (tokens[after] == 299).all()
    assert float((scores - want).abs().max()) <= TOL[dtype] * T
    assert len({tuple(t) for t in tokens[0].tolist()}) == W


def test_one_beam_is_greedy(ex):
    model = ex.Model(vocab=300, width=128, layers=1, dtype=torch.float32, seed=5)
    prompt = torch.randint(0, 300, (2, 20), generator=torch.Generator().manual_seed(0)).cuda()
    tokens, _ = ex.beam_search(model, prompt, 1, 6, eos=299)
    logits, caches = model.prompt(prompt)
    now, got = logits[:, -1].argmax(-1), []
    for t in range(6):
        got.append(now)
        positions = torch.full((2,), 20 + t, dtype=torch.int32, device="cuda")
        now = model.step(now, caches, positions).argmax(-1)
    assert torch.equal(torch.stack(got, 1), tokens[:, 0].long())


def test_command_line(ex, monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["beam_search.py", "--batch", "1", "--beams", "2", "--prompt", "5", "--tokens", "3"])
    ex.main()
    assert "1 requests x 2 beams, 3 tokens" in capsys.readouterr().out
