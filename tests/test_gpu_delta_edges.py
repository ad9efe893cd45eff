"""The gated delta rule in chunks at values where it can go wrong, against the
recurrence in 64 bits (bounds: delta_ref)."""
import pytest
import torch

from test_gpu_delta import inputs, run, ssd  # noqa: F401

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
