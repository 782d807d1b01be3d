"""Parameter and gradient vectors of the norm calls given as addresses: an
address says nothing about its elements, so a type comes from the dtype argument
or from the tensor beside it (weight with bias, dweight with dbias, dw with
dbias), and a call that has neither is refused. Nothing is launched: the calls
that are accepted have no rows."""
import pytest

import gradient_sync_zr_amd as zr
from test_abi_cpu import A

B, C, D, E = (A + (i << 36) for i in range(1, 5))
BF, FP = zr.ZR_BF16, zr.ZR_FP32


def fwd(weight=None, bias=None, **kw):
    zr.zr_layernorm_fwd(A, 0, 64, B, weight, bias, x_dtype=BF, y_dtype=BF, stream=0, **kw)


def bwd(**kw):
    zr.zr_layernorm_bwd(A, B, 0, 64, C, C + 4096, dx=D, dy_dtype=BF, x_dtype=BF, dx_dtype=BF, stream=0, **kw)


@pytest.mark.parametrize("name", ["weight", "bias"])
def test_forward_parameters_need_a_type(name):
    with pytest.raises(ValueError, match=f"{name} is an address: its dtype is needed"):
        fwd(**{name: E})
    for dt in (BF, FP):
        fwd(param_dtype=dt, **{name: E})


def test_backward_parameters_need_a_type():
    with pytest.raises(ValueError, match="weight is an address: its dtype is needed"):
        bwd(weight=E)
    bwd(weight=E, param_dtype=BF)


@pytest.mark.parametrize("name", ["dweight", "dbias"])
def test_gradients_need_a_type(name):
    """(Taken as fp32, a gradient inside a bf16 buffer would be written over its neighbour.)"""
    for kw in ({}, {"accumulate": True}):
        with pytest.raises(ValueError, match=f"{name} is an address: its dtype is needed"):
            bwd(**{name: E}, **kw)
    bwd(accumulate=True, grad_dtype=BF, **{name: E})


def test_the_tensor_beside_an_address_gives_its_type():
    import torch
    # (the tensors are not on a GPU: a call that gets this far is past its dtypes)
    for one, two in ((E, torch.zeros(64, dtype=torch.bfloat16)), (torch.zeros(64), E)):
        with pytest.raises(ValueError, match="not on the GPU"):
            fwd(one, two)
        with pytest.raises(ValueError, match="not on the GPU"):
            bwd(dweight=one, dbias=two)
    with pytest.raises(ValueError, match="not on the GPU"):
        zr.zr_ckpt_wgrad(A, B, 0, 4, 64, torch.zeros(4, 64), dbias=E, dy_dtype=BF, stream=0)


def test_no_vector_needs_no_type():
    fwd()
    fwd(weight=0, bias=0)
    bwd()
    bwd(weight=0, dweight=0, dbias=0)
