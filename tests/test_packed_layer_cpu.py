"""What the packed layer and the clipped optimizer step refuse before they call anything (no GPU)."""
import pytest

from gradient_sync_zr_amd.steps import PackedNormLinear


def layer(**kw):
    import torch
    made = PackedNormLinear(torch.zeros(5000), 0, 8, 40, 50, **kw)
    made._packed = True
    return made


def test_bias_of_the_layer_and_of_the_call_agree():
    """Without, its gradient would be lost, or one of no bias written into the flat gradient."""
    import torch
    x, w, z, b = torch.zeros(8, 40), torch.zeros(40), torch.zeros(8, 50), torch.zeros(50)
    with pytest.raises(ValueError, match="forward has no bias"):
        layer().forward(x, w, z)
    with pytest.raises(ValueError, match="bias=False"):
        layer(bias=False).forward(x, w, z, bias=b)
    for made, bias in ((layer(), b), (layer(bias=False), None)):
        with pytest.raises(ValueError, match="not on the GPU"):  # the call itself
            made.forward(x, w, z, bias=bias)
        assert not made._ran


def test_weight_formats():
    """Of a format that no product takes, a layer would pack its weight, run its norm, and fail there."""
    import gradient_sync_zr_amd as zr
    for good in (zr.ZR_CKPT_E4M3, zr.ZR_CKPT_E2M1):
        layer(weight_format=good)
    for bad in (zr.ZR_CKPT_INT8, zr.ZR_BF16, 9):
        with pytest.raises(ValueError, match="weight_format"):
            layer(weight_format=bad)
