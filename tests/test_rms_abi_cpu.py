"""Refusals of the RMS norm, packing and linear layer calls, without a GPU: every
bad argument is reported before any HIP call (fake addresses, nothing launched)."""
import pytest

import gradient_sync_zr_amd as zr
import pack_ref as pk
from test_abi_cpu import A, expect

B, C, D, E, F, G = (A + (i << 36) for i in range(1, 7))
BF, FP, E4, I8, E2 = zr.ZR_BF16, zr.ZR_FP32, zr.ZR_CKPT_E4M3, zr.ZR_CKPT_INT8, zr.ZR_CKPT_E2M1


def test_constants_agree_with_the_header():
    import os
    import re
    from conftest import ROOT
    text = open(os.path.join(ROOT, "include", "zr.h")).read()
    assert int(re.search(r"\bZR_CKPT_E2M1 = (\d+)", text).group(1)) == E2 == pk.E2M1


@pytest.mark.parametrize("rows,cols", [(0, 1), (1, 1), (1, 32), (7, 33), (100, 4096), (1 << 20, 1 << 20)])
def test_bytes(rows, cols):
    for fmt in (E4, I8, E2):
        assert zr.zr_ckpt_format_bytes(rows, cols, fmt) == pk.nbytes(rows, cols, fmt)
    for fmt in (BF, FP, 5, -1):
        assert zr.zr_ckpt_format_bytes(rows, cols, fmt) == 0


def test_sizes_out_of_range_have_no_bytes():
    for rows, cols in ((-1, 4), (4, 0), (4, -3), (4, (1 << 30) + 1), ((1 << 20) + 1, 1 << 20), (1 << 40, 1)):
        assert zr.zr_ckpt_format_bytes(rows, cols, E2) == 0
        assert zr.zr_rmsnorm_workspace_bytes(rows, cols) == 0
        assert zr.zr_ckpt_linear_workspace_bytes(rows, cols, 8) == 0
        assert zr.zr_ckpt_linear_workspace_bytes(rows, 8, cols) == 0
    assert zr.zr_ckpt_linear_workspace_bytes(0, 100, 100) == 0


def pack(x=A, rows=10, cols=100, ckpt=B, fmt=E2, dt=BF, ld=None):
    zr.zr_ckpt_pack(x, rows, cols, ckpt, format=fmt, dtype=dt, ld=ld, stream=0)


def unpack(x=A, rows=10, cols=100, ckpt=B, fmt=E2, dt=BF, ld=None):
    zr.zr_ckpt_unpack(ckpt, rows, cols, x, format=fmt, dtype=dt, ld=ld, stream=0)


@pytest.mark.parametrize("call", [pack, unpack])
def test_small_blocks_refusals(call):
    for rows, cols in ((-1, 8), (4, 0), (4, (1 << 30) + 1), (1 << 40, 64)):
        expect(zr.ZR_ERR_INVALID, call, rows=rows, cols=cols)
    expect(zr.ZR_ERR_INVALID, call, ld=99)
    expect(zr.ZR_ERR_UNSUPPORTED, call, fmt=5)
    expect(zr.ZR_ERR_UNSUPPORTED, call, dt=E2)
    expect(zr.ZR_ERR_ALIGN, call, ckpt=B + 8)
    expect(zr.ZR_ERR_ALIAS, call, x=B + 10 * 68 - 4)      # x starts in the buffer's last bytes
    call(rows=0, x=0, ckpt=0)


def pack_t(x=A, rows=10, cols=100, ckpt=B, fmt=E4, dt=BF, ld=None):
    zr.zr_ckpt_pack_t(x, rows, cols, ckpt, format=fmt, dtype=dt, ld=ld, stream=0)


def test_transposed_pack_refusals():
    for rows, cols in ((-1, 8), (0, 8), (4, 0), (4, (1 << 30) + 1), ((1 << 30) + 1, 4), (1 << 25, 1 << 20)):
        expect(zr.ZR_ERR_INVALID, pack_t, rows=rows, cols=cols)
    expect(zr.ZR_ERR_INVALID, pack_t, ld=99)
    expect(zr.ZR_ERR_UNSUPPORTED, pack_t, fmt=BF)
    expect(zr.ZR_ERR_UNSUPPORTED, pack_t, dt=E4)
    expect(zr.ZR_ERR_INVALID, pack_t, x=0)
    expect(zr.ZR_ERR_ALIGN, pack_t, ckpt=B + 4)
    expect(zr.ZR_ERR_ALIAS, pack_t, x=B + 100 * 33 - 2)   # 100 rows of one block
    expect(zr.ZR_ERR_ALIAS, pack_t, ckpt=A + 16)


def fwd(**kw):
    a = dict(x=A, rows=10, cols=100, y=B, weight=C, residual=D, h=E, x_dtype=BF, y_dtype=BF, h_dtype=BF, param_dtype=BF,
             stream=0)
    a.update(kw)
    zr.zr_rmsnorm_fwd(**a)


def test_forward_refusals():
    for rows, cols in ((-1, 8), (4, 0), (4, (1 << 30) + 1), (1 << 40, 64)):
        expect(zr.ZR_ERR_INVALID, fwd, rows=rows, cols=cols)
    for eps in (-1e-5, float("nan"), float("inf")):
        expect(zr.ZR_ERR_INVALID, fwd, eps=eps)
    expect(zr.ZR_ERR_INVALID, fwd, x=0)
    expect(zr.ZR_ERR_INVALID, fwd, y=None, h=None)
    expect(zr.ZR_ERR_INVALID, fwd, residual=None)         # h would be x
    expect(zr.ZR_ERR_INVALID, fwd, x_dtype=E4, residual=None, h=None, ckpt_h=F)
    for n in ("ld_x", "ld_y", "ld_h", "ld_residual"):
        expect(zr.ZR_ERR_INVALID, fwd, **{n: 99})
    for n in ("y_dtype", "h_dtype", "param_dtype"):
        expect(zr.ZR_ERR_UNSUPPORTED, fwd, **{n: E4})
    expect(zr.ZR_ERR_UNSUPPORTED, fwd, x_dtype=E2)
    expect(zr.ZR_ERR_UNSUPPORTED, fwd, ckpt_y=F, ckpt_format=E2)
    expect(zr.ZR_ERR_ALIGN, fwd, x=A + 1)
    expect(zr.ZR_ERR_ALIGN, fwd, rstd=F + 2)
    expect(zr.ZR_ERR_ALIGN, fwd, ckpt_h=F + 4)
    expect(zr.ZR_ERR_ALIAS, fwd, h=B)
    expect(zr.ZR_ERR_ALIAS, fwd, h=A + 2)
    expect(zr.ZR_ERR_ALIAS, fwd, h=A, ld_h=101)
    expect(zr.ZR_ERR_ALIAS, fwd, y=D, y_dtype=FP)
    expect(zr.ZR_ERR_ALIAS, fwd, h=D, y=D)
    expect(zr.ZR_ERR_ALIAS, fwd, y=C)
    expect(zr.ZR_ERR_ALIAS, fwd, ckpt_h=F, ckpt_y=F + 16)
    expect(zr.ZR_ERR_ALIAS, fwd, x_dtype=E4, h=A)
    fwd(rows=0)
    fwd(rows=0, x=0, y=0, h=0, residual=0)


def bwd(**kw):
    a = dict(dy=A, h=B, rows=300, cols=100, rstd=C, weight=D, dx=E, dweight=F, workspace=(G, 1 << 30), dy_dtype=BF,
             h_dtype=BF, dx_dtype=BF, param_dtype=BF, grad_dtype=FP, stream=0)
    a.update(kw)
    zr.zr_rmsnorm_bwd(**a)


def test_backward_refusals():
    for rows, cols in ((-1, 8), (4, 0), (4, (1 << 30) + 1), (1 << 40, 64)):
        expect(zr.ZR_ERR_INVALID, bwd, rows=rows, cols=cols)
    for n in ("dy", "h", "rstd"):
        expect(zr.ZR_ERR_INVALID, bwd, **{n: 0})
    expect(zr.ZR_ERR_INVALID, bwd, dx=None, dweight=None)
    for n in ("ld_dy", "ld_h", "ld_dx"):
        expect(zr.ZR_ERR_INVALID, bwd, **{n: 99})
    for n in ("dy_dtype", "param_dtype", "dx_dtype", "grad_dtype"):
        expect(zr.ZR_ERR_UNSUPPORTED, bwd, **{n: E4})
    expect(zr.ZR_ERR_UNSUPPORTED, bwd, h_dtype=E2)
    need = zr.zr_rmsnorm_workspace_bytes(300, 100)
    assert need > 0
    expect(zr.ZR_ERR_WORKSPACE, bwd, workspace=None)
    expect(zr.ZR_ERR_WORKSPACE, bwd, workspace=(G, need - 1))
    expect(zr.ZR_ERR_ALIGN, bwd, workspace=(G + 2, need))
    expect(zr.ZR_ERR_ALIGN, bwd, dweight=F + 2)
    expect(zr.ZR_ERR_ALIAS, bwd, workspace=(E, need))
    expect(zr.ZR_ERR_ALIAS, bwd, dx=A + 2)
    expect(zr.ZR_ERR_ALIAS, bwd, dx=A, dx_dtype=FP)
    expect(zr.ZR_ERR_ALIAS, bwd, dx=B, h_dtype=E4)
    expect(zr.ZR_ERR_ALIAS, bwd, dx=A, rows=1, dx_dtype=FP)
    expect(zr.ZR_ERR_ALIAS, bwd, dweight=C)
    bwd(rows=0, dweight=None, workspace=None)
    bwd(rows=0, accumulate=True, workspace=None)
    lib = zr.lib()
    for flags in (1, 8, -1):
        assert lib.zr_rmsnorm_bwd(A, BF, 100, B, BF, 100, 10, 100, D, BF, C, E, BF, 100, F, FP, flags, G, 1 << 30,
                                  None) == zr.ZR_ERR_INVALID


def linear(**kw):
    a = dict(x=A, w=B, rows=200, in_cols=4096, out_cols=70, z=C, bias=D, x_format=E4, w_format=E2, z_dtype=BF, bias_dtype=FP,
             workspace=(E, 1 << 30), stream=0)
    a.update(kw)
    zr.zr_ckpt_linear(**a)


def test_linear_refusals():
    for k in ("out_cols", "in_cols"):
        for v in (0, -1, (1 << 30) + 1):
            expect(zr.ZR_ERR_INVALID, linear, **{k: v})
    expect(zr.ZR_ERR_INVALID, linear, rows=-1)
    expect(zr.ZR_ERR_INVALID, linear, rows=1 << 40)
    expect(zr.ZR_ERR_INVALID, linear, ld_z=69)
    for n in ("x", "w", "z"):
        expect(zr.ZR_ERR_INVALID, linear, **{n: 0})
    for n in ("x_format", "w_format"):
        for bad in (I8, BF, 9):
            expect(zr.ZR_ERR_UNSUPPORTED, linear, **{n: bad})
    expect(zr.ZR_ERR_UNSUPPORTED, linear, z_dtype=E4)
    expect(zr.ZR_ERR_UNSUPPORTED, linear, bias_dtype=E4)
    need = zr.zr_ckpt_linear_workspace_bytes(200, 4096, 70)
    assert need > 0
    expect(zr.ZR_ERR_WORKSPACE, linear, workspace=None)
    expect(zr.ZR_ERR_WORKSPACE, linear, workspace=(E, need - 1))
    expect(zr.ZR_ERR_ALIGN, linear, workspace=(E + 2, need))
    expect(zr.ZR_ERR_ALIGN, linear, x=A + 8)
    expect(zr.ZR_ERR_ALIGN, linear, z=C + 1)
    expect(zr.ZR_ERR_ALIGN, linear, bias=D + 2)
    expect(zr.ZR_ERR_ALIAS, linear, z=A)
    expect(zr.ZR_ERR_ALIAS, linear, z=B + 70 * 2176 - 2)  # the weight's last exponents, 4-bit rows
    expect(zr.ZR_ERR_ALIAS, linear, z=D)
    expect(zr.ZR_ERR_ALIAS, linear, workspace=(C, need))
    linear(rows=0, x=0, z=0, workspace=None)
    lib = zr.lib()
    for flags in (1, 4, 8, -1):
        assert lib.zr_ckpt_linear(A, E4, B, E4, 10, 64, 70, None, BF, C, BF, 70, flags, E, 1 << 30, None) == zr.ZR_ERR_INVALID


def test_tensors_are_checked():
    import torch
    x = torch.zeros(zr.zr_ckpt_format_bytes(4, 64, E2), dtype=torch.uint8)
    with pytest.raises(ValueError, match="zr_ckpt_format_bytes"):
        zr.zr_ckpt_linear(x[:-1], B, 4, 64, 8, C, x_format=E2, z_dtype=BF, stream=0)
    with pytest.raises(ValueError, match="zr_ckpt_bytes"):
        zr.zr_ckpt_linear(x, B, 4, 64, 8, C, z_dtype=BF, stream=0)     # e4m3 needs more
    with pytest.raises(ValueError, match="not on the GPU"):
        zr.zr_ckpt_linear(x, B, 4, 64, 8, C, x_format=E2, z_dtype=BF, stream=0)
    with pytest.raises(ValueError, match="its dtype is needed"):
        zr.zr_ckpt_linear(A, B, 4, 64, 8, C, bias=D, z_dtype=BF, stream=0)
    with pytest.raises(ValueError, match="different dtypes"):
        zr.zr_rmsnorm_fwd(A, 4, 64, residual=torch.zeros(4, 64), h=torch.zeros(4, 64).bfloat16(), x_dtype=BF, stream=0)
