"""Refusals of the layer norm and checkpoint calls, without a GPU: every bad
argument is reported before any HIP call (fake addresses, nothing launched)."""
import ctypes

import pytest

import gradient_sync_zr_amd as zr
import ckpt_ref as ref
from test_abi_cpu import A, expect

B, C, D, E, F, G = (A + (i << 36) for i in range(1, 7))
BF, FP = zr.ZR_BF16, zr.ZR_FP32


def test_constants_agree_with_the_header():
    import os
    import re
    from conftest import ROOT
    text = open(os.path.join(ROOT, "include", "zr.h")).read()
    for n in ("ZR_CKPT_E4M3", "ZR_CKPT_INT8"):
        assert int(re.search(rf"\b{n} = (\d+)", text).group(1)) == getattr(zr, n)
    assert int(re.search(r"#define ZR_ADD_DX (\d+)", text).group(1)) == zr.ZR_ADD_DX


@pytest.mark.parametrize("rows,cols", [(0, 1), (1, 1), (1, 32), (7, 33), (100, 4096), (1 << 20, 1 << 20), (1 << 10, 1 << 30)])
def test_checkpoint_bytes(rows, cols):
    assert zr.zr_ckpt_bytes(rows, cols) == ref.nbytes(rows, cols)


def test_sizes_out_of_range_have_no_bytes():
    for rows, cols in ((-1, 4), (4, 0), (4, -3), (4, (1 << 30) + 1), ((1 << 20) + 1, 1 << 20), (1 << 40, 1)):
        assert zr.zr_ckpt_bytes(rows, cols) == 0
        assert zr.zr_layernorm_workspace_bytes(rows, cols) == 0
        assert zr.zr_ckpt_wgrad_workspace_bytes(rows, 8, cols) == 0
        assert zr.zr_ckpt_wgrad_workspace_bytes(rows, cols, 8) == 0


def pack(x=A, rows=10, cols=100, ckpt=B, fmt=zr.ZR_CKPT_E4M3, dt=BF, ld=None):
    zr.zr_ckpt_pack(x, rows, cols, ckpt, format=fmt, dtype=dt, ld=ld, stream=0)


def unpack(x=A, rows=10, cols=100, ckpt=B, fmt=zr.ZR_CKPT_E4M3, dt=BF, ld=None):
    zr.zr_ckpt_unpack(ckpt, rows, cols, x, format=fmt, dtype=dt, ld=ld, stream=0)


@pytest.mark.parametrize("call", [pack, unpack])
def test_pack_and_unpack_refusals(call):
    for rows, cols in ((-1, 8), (4, 0), (4, -1), (4, (1 << 30) + 1), (1 << 40, 64)):
        expect(zr.ZR_ERR_INVALID, call, rows=rows, cols=cols)
    expect(zr.ZR_ERR_INVALID, call, ld=99)
    expect(zr.ZR_ERR_INVALID, call, rows=1 << 20, ld=(1 << 20) + 1)
    expect(zr.ZR_ERR_UNSUPPORTED, call, fmt=BF)
    expect(zr.ZR_ERR_UNSUPPORTED, call, fmt=7)
    expect(zr.ZR_ERR_UNSUPPORTED, call, dt=zr.ZR_CKPT_INT8)
    expect(zr.ZR_ERR_INVALID, call, x=0)
    expect(zr.ZR_ERR_INVALID, call, ckpt=0)
    expect(zr.ZR_ERR_ALIGN, call, x=A + 1)
    expect(zr.ZR_ERR_ALIGN, call, dt=FP, x=A + 2)
    expect(zr.ZR_ERR_ALIGN, call, ckpt=B + 8)
    expect(zr.ZR_ERR_ALIAS, call, ckpt=A + 64)
    expect(zr.ZR_ERR_ALIAS, call, x=B + 10 * 132 - 4)     # x starts in the checkpoint's last bytes
    call(rows=0)                                          # no work
    call(rows=0, x=0, ckpt=0)


def fwd(**kw):
    a = dict(x=A, rows=10, cols=100, y=B, weight=C, bias=D, x_dtype=BF, y_dtype=BF, param_dtype=BF, stream=0)
    a.update(kw)
    zr.zr_layernorm_fwd(**a)


def test_forward_refusals():
    for rows, cols in ((-1, 8), (4, 0), (4, (1 << 30) + 1), (1 << 40, 64)):
        expect(zr.ZR_ERR_INVALID, fwd, rows=rows, cols=cols)
    for eps in (-1e-5, float("nan"), float("inf")):
        expect(zr.ZR_ERR_INVALID, fwd, eps=eps)
    expect(zr.ZR_ERR_INVALID, fwd, x=0)
    expect(zr.ZR_ERR_INVALID, fwd, y=None)
    expect(zr.ZR_ERR_INVALID, fwd, ld_x=99)
    expect(zr.ZR_ERR_INVALID, fwd, ld_y=99)
    expect(zr.ZR_ERR_UNSUPPORTED, fwd, x_dtype=9)
    expect(zr.ZR_ERR_UNSUPPORTED, fwd, y_dtype=zr.ZR_CKPT_E4M3)
    expect(zr.ZR_ERR_UNSUPPORTED, fwd, param_dtype=zr.ZR_CKPT_INT8)
    expect(zr.ZR_ERR_UNSUPPORTED, fwd, ckpt_y=E, ckpt_format=BF)
    expect(zr.ZR_ERR_INVALID, fwd, x_dtype=zr.ZR_CKPT_E4M3, ckpt_x=E)   # x is one already
    expect(zr.ZR_ERR_ALIGN, fwd, x=A + 1)
    expect(zr.ZR_ERR_ALIGN, fwd, x_dtype=zr.ZR_CKPT_E4M3, x=A + 2)
    expect(zr.ZR_ERR_ALIGN, fwd, mean=E + 2)
    expect(zr.ZR_ERR_ALIGN, fwd, ckpt_x=E + 4)
    expect(zr.ZR_ERR_ALIGN, fwd, weight=C + 1)
    expect(zr.ZR_ERR_ALIAS, fwd, y=A + 2)                 # shifted in place
    expect(zr.ZR_ERR_ALIAS, fwd, y=A, y_dtype=FP)         # in place, other type
    expect(zr.ZR_ERR_ALIAS, fwd, y=A, ld_y=101)
    expect(zr.ZR_ERR_ALIAS, fwd, y=C)
    expect(zr.ZR_ERR_ALIAS, fwd, mean=E, rstd=E + 36)
    expect(zr.ZR_ERR_ALIAS, fwd, ckpt_x=E, ckpt_y=E + 16)
    expect(zr.ZR_ERR_ALIAS, fwd, ckpt_x=A)
    expect(zr.ZR_ERR_ALIAS, fwd, y=A + 100, ld_x=128, ld_y=128)   # columns 50.. of the same wide rows
    fwd(rows=0)
    fwd(rows=0, x=0, y=B)


def bwd(**kw):
    a = dict(dy=A, x=B, rows=300, cols=100, mean=C, rstd=C + 4096, weight=D, dx=E, dweight=F, dbias=F + 4096,
             workspace=(G, 1 << 30), dy_dtype=BF, x_dtype=BF, dx_dtype=BF, param_dtype=BF, grad_dtype=FP, stream=0)
    a.update(kw)
    zr.zr_layernorm_bwd(**a)


def test_backward_refusals():
    for rows, cols in ((-1, 8), (4, 0), (4, (1 << 30) + 1), (1 << 40, 64)):
        expect(zr.ZR_ERR_INVALID, bwd, rows=rows, cols=cols)
    for n in ("dy", "x", "mean", "rstd"):
        expect(zr.ZR_ERR_INVALID, bwd, **{n: 0})
    expect(zr.ZR_ERR_INVALID, bwd, dx=None, dweight=None, dbias=None)
    for n in ("ld_dy", "ld_x", "ld_dx"):
        expect(zr.ZR_ERR_INVALID, bwd, **{n: 99})
    for n in ("dy_dtype", "param_dtype", "dx_dtype", "grad_dtype"):
        expect(zr.ZR_ERR_UNSUPPORTED, bwd, **{n: zr.ZR_CKPT_E4M3})
    expect(zr.ZR_ERR_UNSUPPORTED, bwd, x_dtype=11)
    need = zr.zr_layernorm_workspace_bytes(300, 100)
    assert need > 0
    expect(zr.ZR_ERR_WORKSPACE, bwd, workspace=None)
    expect(zr.ZR_ERR_WORKSPACE, bwd, workspace=(G, need - 1))
    expect(zr.ZR_ERR_ALIGN, bwd, workspace=(G + 2, need))
    expect(zr.ZR_ERR_ALIGN, bwd, dweight=F + 2)
    expect(zr.ZR_ERR_ALIGN, bwd, dx=E + 1)
    expect(zr.ZR_ERR_ALIAS, bwd, dbias=F + 396)
    expect(zr.ZR_ERR_ALIAS, bwd, workspace=(E, need))
    expect(zr.ZR_ERR_ALIAS, bwd, workspace=(A, need))
    expect(zr.ZR_ERR_ALIAS, bwd, dx=A + 2)
    expect(zr.ZR_ERR_ALIAS, bwd, dx=A, dx_dtype=FP)
    expect(zr.ZR_ERR_ALIAS, bwd, dx=A, ld_dx=128)
    expect(zr.ZR_ERR_ALIAS, bwd, dx=B, x_dtype=zr.ZR_CKPT_E4M3)
    expect(zr.ZR_ERR_ALIAS, bwd, dx=A, rows=1, dx_dtype=FP)
    expect(zr.ZR_ERR_ALIAS, bwd, dweight=C)
    bwd(rows=0, dweight=None, dbias=None, workspace=None)
    lib = zr.lib()
    for flags in (1, 8, -1):
        assert lib.zr_layernorm_bwd(A, BF, 100, B, BF, 100, 10, 100, D, BF, C, C + 4096, E, BF, 100, F, F + 4096, FP,
                                    flags, G, 1 << 30, None) == zr.ZR_ERR_INVALID


def wgrad(**kw):
    a = dict(dy=A, ckpt=B, rows=8192, out_cols=100, in_cols=70, dw=C, dbias=D, workspace=(E, 1 << 30), dy_dtype=BF,
             grad_dtype=FP, stream=0)
    a.update(kw)
    zr.zr_ckpt_wgrad(**a)


def test_wgrad_refusals():
    for k in ("out_cols", "in_cols"):
        for v in (0, -1, (1 << 30) + 1):
            expect(zr.ZR_ERR_INVALID, wgrad, **{k: v})
    expect(zr.ZR_ERR_INVALID, wgrad, rows=-1)
    expect(zr.ZR_ERR_INVALID, wgrad, rows=1 << 40)
    expect(zr.ZR_ERR_INVALID, wgrad, ld_dy=99)
    expect(zr.ZR_ERR_INVALID, wgrad, ld_dw=69)
    for n in ("dy", "ckpt", "dw"):
        expect(zr.ZR_ERR_INVALID, wgrad, **{n: 0})
    expect(zr.ZR_ERR_UNSUPPORTED, wgrad, dy_dtype=zr.ZR_CKPT_E4M3)
    expect(zr.ZR_ERR_UNSUPPORTED, wgrad, grad_dtype=zr.ZR_CKPT_E4M3, dbias=None)
    expect(zr.ZR_ERR_UNSUPPORTED, wgrad, format=BF)
    need = zr.zr_ckpt_wgrad_workspace_bytes(8192, 100, 70)
    assert need > 0
    expect(zr.ZR_ERR_WORKSPACE, wgrad, workspace=None)
    expect(zr.ZR_ERR_WORKSPACE, wgrad, workspace=(E, need - 1))
    expect(zr.ZR_ERR_ALIGN, wgrad, workspace=(E + 2, need))
    expect(zr.ZR_ERR_ALIGN, wgrad, ckpt=B + 8)
    expect(zr.ZR_ERR_ALIGN, wgrad, dw=C + 2)
    expect(zr.ZR_ERR_ALIAS, wgrad, dbias=C + 4 * 6999)
    expect(zr.ZR_ERR_ALIAS, wgrad, dw=B)
    expect(zr.ZR_ERR_ALIAS, wgrad, workspace=(C, need))
    lib = zr.lib()
    for flags in (1, 4, 8, -1):
        assert lib.zr_ckpt_wgrad(A, BF, 100, B, zr.ZR_CKPT_E4M3, 256, 100, 70, C, FP, 70, D, flags, E, 1 << 30,
                                 None) == zr.ZR_ERR_INVALID


def test_null_pointers_through_the_c_call():
    lib = zr.lib()
    assert lib.zr_ckpt_pack(None, BF, 4, 8, 8, ctypes.c_void_p(A), zr.ZR_CKPT_E4M3, None) == zr.ZR_ERR_INVALID
    assert "x is NULL" in zr.zr_last_error()


def test_tensors_are_checked():
    import torch
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    ck = torch.zeros(zr.zr_ckpt_bytes(4, 64), dtype=torch.uint8)
    with pytest.raises(ValueError, match="not on the GPU"):
        zr.zr_ckpt_pack(x, 4, 64, ck, stream=0)
    for bad, why in ((dict(rows=5), "5 x 64"), (dict(x=x.t(), rows=64, cols=4), "not contiguous"),
                     (dict(dtype=torch.float32), "dtype"), (dict(ld=65), "row stride"), (dict(x=x.int()), "unsupported dtype")):
        a = dict(x=x, rows=4, cols=64, ckpt=A, stream=0)
        a.update(bad)
        with pytest.raises((ValueError, TypeError), match=why):
            zr.zr_ckpt_pack(**a)
    for ckpt in (ck[:-1], ck.view(torch.int16), torch.zeros(2 * ck.numel(), dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="zr_ckpt_bytes"):
            zr.zr_ckpt_pack(A, 4, 64, ckpt, dtype=BF, stream=0)
    with pytest.raises(ValueError, match="its dtype is needed"):
        zr.zr_ckpt_pack(A, 4, 64, B, stream=0)
    w = torch.zeros(63)
    with pytest.raises(ValueError, match="weight is not 64"):
        zr.zr_layernorm_fwd(A, 4, 64, B, w, x_dtype=BF, y_dtype=BF, stream=0)
    with pytest.raises(ValueError, match="different dtypes"):
        zr.zr_layernorm_fwd(A, 4, 64, B, torch.zeros(64), torch.zeros(64, dtype=torch.bfloat16), x_dtype=BF, y_dtype=BF,
                            stream=0)
    with pytest.raises(ValueError, match="mean is torch.float64|dtype"):
        zr.zr_layernorm_fwd(A, 4, 64, B, mean=torch.zeros(4, dtype=torch.bfloat16), x_dtype=BF, y_dtype=BF, stream=0)
