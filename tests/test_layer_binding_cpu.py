"""CPU tests of what the layer operators' binding refuses or does by itself, before any call reaches
the library's validation."""
import pytest
import torch

from mxfp8_block_scaled_partial_amd import layer as L

OTHERS = [torch.int8, torch.bool, torch.float8_e5m2, torch.float8_e4m3fnuz, torch.int16, torch.float32]


@pytest.mark.parametrize("dtype", OTHERS + [torch.float8_e8m0fnu], ids=str)
def test_codes_of_another_format_are_refused(dtype):
    data, scale = torch.zeros(64, 256).to(dtype), torch.zeros(64, 2, dtype=torch.uint8)
    with pytest.raises(ValueError, match="data must be uint8 or torch.float8_e4m3fn"):
        L.make_operand(data, scale)
    with pytest.raises(ValueError, match=r"row\[0\] data must be uint8 or torch.float8_e4m3fn"):
        L._mat8((data, scale), 64, 256, False, "row[0]")


@pytest.mark.parametrize("dtype", OTHERS + [torch.float8_e4m3fn], ids=str)
def test_scales_of_another_format_are_refused(dtype):
    data, scale = torch.zeros(64, 256, dtype=torch.uint8), torch.zeros(64, 2).to(dtype)
    with pytest.raises(ValueError, match="scale must be uint8 or torch.float8_e8m0fnu"):
        L.make_operand(data, scale)
    with pytest.raises(ValueError, match=r"row\[0\] scale must be uint8 or torch.float8_e8m0fnu"):
        L._mat8((data, scale), 64, 256, False, "row[0]")


def test_views_of_the_right_format_are_taken():
    """The next check is then that they lie on the device."""
    data, scale = torch.zeros(64, 256, dtype=torch.uint8), torch.ones(64, 2, dtype=torch.uint8)
    for d in (data, data.view(torch.float8_e4m3fn)):
        for s in (scale, scale.view(torch.float8_e8m0fnu)):
            with pytest.raises(ValueError, match="device tensor"):
                L.make_operand(d, s)
            with pytest.raises(ValueError, match="device tensor"):
                L._mat8((d, s), 64, 256, False, "row[0]")
