"""Arguments of the layer operators at the edge of what they take, without a GPU."""
import pytest
import torch

from test_layer_cpu import ext  # noqa: F401  (fixture)


@pytest.mark.parametrize("code", [-1, 16, 255])
def test_codes_outside_four_bits_are_refused(ext, code):  # noqa: F811
    """Such a code would change its neighbours in the packed word."""
    codes = torch.full((20, 70), 15)
    codes[3, 64] = code
    with pytest.raises(ext.SSDError, match="0 to 15"):
        ext.w4_pack(codes)


def test_packing_nothing(ext):  # noqa: F811
    assert ext.w4_pack(torch.zeros(0, 5, dtype=torch.uint8)).shape == (0, 1, 32, 4)
