"""Arguments of the layer operators at the edge of what they take, without a GPU."""
import pytest
import torch

from test_layer_cpu import ext, step_args, w4_args  # noqa: F401  (ext: fixture)


@pytest.mark.parametrize("code", [-1, 16, 255])
def test_codes_outside_four_bits_are_refused(ext, code):  # noqa: F811
    """Such a code would change its neighbours in the packed word."""
    codes = torch.full((20, 70), 15)
    codes[3, 64] = code
    with pytest.raises(ext.SSDError, match="0 to 15"):
        ext.w4_pack(codes)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_weights_that_are_not_finite_are_refused(ext, bad):  # noqa: F811
    weight = torch.randn(5, 100)
    weight[2, 70] = bad
    with pytest.raises(ext.SSDError, match="finite"):
        ext.w4_quantize(weight, 32)


@pytest.mark.parametrize("weight", [torch.zeros(4), torch.zeros(2, 3, 4)])
def test_weights_that_are_no_matrix_are_refused(ext, weight):  # noqa: F811
    with pytest.raises(ext.SSDError, match="2-D"):
        ext.w4_quantize(weight, 32)


def test_packing_nothing(ext):  # noqa: F811
    assert ext.w4_pack(torch.zeros(0, 5, dtype=torch.uint8)).shape == (0, 1, 32, 4)


@pytest.mark.parametrize("big", [dict(n=2 ** 31 - 1), dict(n=2 ** 30 + 1), dict(k=2 ** 30 + 1)])
def test_products_of_sizes_past_32_bits_are_refused(ext, big):  # noqa: F811
    """Row tiles and rows are counted in 32 bits.  (Refused before anything is looked at.)"""
    assert ext.lib.ssd_w4_matvec(w4_args(ext, **big, x=0, y=0, packed=0), None) == 2


@pytest.mark.parametrize("width,groups", [(4, 2 ** 20), (3, 3 * 2 ** 19), (2, 2 ** 21)])
def test_step_rings_past_32_bits_are_refused(ext, width, groups):  # noqa: F811
    """Offsets within a ring's row of width * channels are 32 bits: 576 channels a head here."""
    args = dict(nheads=groups, ngroups=groups, dstate=256, width=width)
    assert width * groups * 576 >= 2 ** 31
    assert ext.lib.ssd_step(step_args(ext, **args, u=0, ring=0, state=0), None) == 2
    most = (2 ** 31 - 1) // (width * 576)
    assert ext.lib.ssd_step(step_args(ext, **{**args, "nheads": most, "ngroups": most}, u=0, ring=0, state=0), None) == 1
