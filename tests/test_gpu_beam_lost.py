"""Beam selection where every candidate that is left scores minus infinity."""
import pytest
import torch

import layer_ref as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
INF = float("inf")


@pytest.fixture(scope="module")
def ssd():
    import mamba_ssd_forward_chunked_gb300 as m
    return m


def same_choice(got, want, where):
    best, parents, tokens = (t.cpu() for t in got)
    r, rp, rt = want
    assert torch.equal(parents.long(), rp) and torch.equal(tokens.long(), rt), where
    fine = torch.isfinite(r)
    assert torch.equal(torch.isfinite(best), fine), where
    # the log-sum-exp and two additions: EPS of each term
    assert ((best.double() - r).abs()[fine] <= ref.EPS * (r.abs()[fine] + 32)).all(), where


def lost(B, W, V, end, few, dtype):
    """Rows masked but for `few` indexes before `end`, in beams that are lost each in another way."""
    x = torch.full((B, W, V), -INF, dtype=dtype)
    x[:, :, end - few:end] = torch.arange(few, dtype=F32).to(dtype)
    s = torch.full((B, W), -INF)
    s[1::3], x[1::3, :, V - 2] = -1.0, float("nan")
    s[2::3], x[2::3, :, V - 2] = -1.0, INF
    return x, s


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
# rows of one piece, of several short ones, and of two long ones; what is not masked lies in the first
@pytest.mark.parametrize("B,W,V,end", [(3, 1, 200, 190), (3, 2, 5000, 2000), (162, 4, 20000, 16000)],
                         ids=["one", "short", "long"])
@pytest.mark.parametrize("few,k", [(2, 2), (2, 3), (3, 3), (4, 5), (5, 5), (30, 40)])
def test_lost_beams_fall_by_index(ssd, dtype, B, W, V, end, few, k):
    x, s = lost(B, W, V, end, few, dtype)
    same_choice(ssd.ssd_beam_select(x.cuda(), s.cuda(), k), ref.beam(x, s, k), "all lost")
    if W > 1:  # a live beam with fewer candidates than asked for, behind lost ones
        x[:, -1, V - 2], s[:, -1] = -INF, -2.0
        same_choice(ssd.ssd_beam_select(x.cuda(), s.cuda(), k), ref.beam(x, s, k), "one live")
        done = torch.zeros(B, W, dtype=torch.bool)
        done[:, 0] = True
        same_choice(ssd.ssd_beam_select(x.cuda(), s.cuda(), k, finished=done.cuda(), eos=V - 1),
                    ref.beam(x, s, k, done, V - 1), "finished")
