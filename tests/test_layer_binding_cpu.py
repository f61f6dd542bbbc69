"""CPU tests of what the layer operators' binding refuses or does by itself, before any call reaches
the library's validation."""
import pytest
import torch

from mxfp8_block_scaled_partial_amd import binding as B
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


def test_own_workspace_on_another_stream(monkeypatch):
    """The allocator is told, once, of every stream but the workspace's own that a call uses it on; a
    caller's workspace is the caller's to keep."""
    class Library:
        mxfp8_matmul_workspace = mxfp8_layernorm_workspace = staticmethod(lambda p: 64)
        mxfp8_matmul = mxfp8_layernorm_backward = staticmethod(lambda p, stream: 0)

    current, told = [7], []
    monkeypatch.setattr(L, "lib", Library)
    monkeypatch.setattr(B, "_dev_ptr", lambda t, what: None if t is None else 4096)
    monkeypatch.setattr(B, "_stream", lambda s: current[0] if s is None else s)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: handle)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: told.append((t.numel(), s)))
    codes, scale = torch.zeros(8, 128, dtype=torch.uint8), torch.zeros(8, 1, dtype=torch.uint8)
    v = torch.zeros(8)

    def product(**kw):
        return L.make_product(L.make_operand(codes, scale), L.make_operand(codes, scale), torch.zeros(8, 8), **kw)

    def norm(**kw):
        x = torch.zeros(8, 8)
        return L.make_layernorm(x, mean=v, rstd=v, dy=x, dgamma=v, **kw)

    for make, call in ((product, L.mxfp8_matmul), (norm, L.mxfp8_layernorm_backward)):
        told.clear()
        p = make()
        call(p)
        assert told == []
        call(p, stream=9)
        call(p, stream=9)
        call(p, stream=7)
        assert told == [(64, 9)]
        current[0] = 11  # another current stream
        call(p)
        current[0] = 7
        assert told == [(64, 9), (64, 11)]
        call(make(workspace=torch.zeros(64, dtype=torch.uint8)), stream=9)
        assert len(told) == 2
