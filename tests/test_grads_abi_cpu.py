"""Refusals of the gradient norm, scaling and AdamW calls, without a GPU: every
bad argument is reported before any HIP call (fake addresses, nothing launched)."""
import ctypes

import pytest

import gradient_sync_zr_amd as zr
from test_abi_cpu import A, expect

BF, FP = zr.ZR_BF16, zr.ZR_FP32
FAR = 1 << 36
B, C, D, E, F, G = (A + i * FAR for i in range(1, 7))
GAP = 1 << 24


def at(base, n=3):
    return [base + i * GAP for i in range(n)]


def norm(grads=None, numels=(10, 0, 1000), norm=B, coef=B + 4, ws=(C, 1 << 20), dt=FP, **kw):
    zr.zr_grad_norm(at(A) if grads is None else grads, numels, norm, coef, workspace=ws, dtype=dt, stream=0, **kw)


def test_norm_refusals():
    for bad in (0.0, -1.0, float("nan"), float("inf"), 1e39):
        expect(zr.ZR_ERR_INVALID, norm, scale=bad)
    for bad in (0.0, -1.0, float("nan")):
        expect(zr.ZR_ERR_INVALID, norm, max_norm=bad)
    expect(zr.ZR_ERR_INVALID, norm, norm=None, coef=None)
    expect(zr.ZR_ERR_INVALID, norm, numels=(10, -1, 4))
    expect(zr.ZR_ERR_INVALID, norm, numels=(10, 1 << 40, 4))
    expect(zr.ZR_ERR_INVALID, norm, grads=[A, B, 0])
    expect(zr.ZR_ERR_UNSUPPORTED, norm, dt=zr.ZR_CKPT_E4M3)
    expect(zr.ZR_ERR_ALIGN, norm, grads=[A, B, A + FAR // 2 + 2])
    expect(zr.ZR_ERR_ALIGN, norm, norm=B + 2)
    expect(zr.ZR_ERR_ALIGN, norm, ws=(C + 4, 1 << 20))
    need = zr.zr_grad_norm_workspace_bytes(3)
    assert need > 0 and zr.zr_grad_norm_workspace_bytes(0) == 0 and zr.zr_grad_norm_workspace_bytes(-3) == 0
    assert zr.zr_grad_norm_workspace_bytes(192) == need and zr.zr_grad_norm_workspace_bytes(193) == 2 * need
    expect(zr.ZR_ERR_WORKSPACE, norm, ws=None)
    expect(zr.ZR_ERR_WORKSPACE, norm, ws=(C, need - 1))
    expect(zr.ZR_ERR_ALIAS, norm, coef=B)
    expect(zr.ZR_ERR_ALIAS, norm, norm=A + 36)
    expect(zr.ZR_ERR_ALIAS, norm, ws=(A + 2 * GAP + 3992, need))
    expect(zr.ZR_ERR_ALIAS, norm, ws=(B - need + 8, need))
    with pytest.raises(ValueError, match="entries"):
        norm(numels=(10, 20))
    with pytest.raises(ValueError, match="dtype is needed"):
        norm(dt=None)
    lib = zr.lib()
    n = (ctypes.c_int64 * 1)(5)
    assert lib.zr_grad_norm(-1, None, None, FP, 1.0, 1.0, B, None, C, 1 << 20, None) == zr.ZR_ERR_INVALID
    assert lib.zr_grad_norm(1, None, n, FP, 1.0, 1.0, B, None, C, 1 << 20, None) == zr.ZR_ERR_INVALID
    assert lib.zr_grad_norm(1, zr.table([A]), None, FP, 1.0, 1.0, B, None, C, 1 << 20, None) == zr.ZR_ERR_INVALID


def scale(grads=None, numels=(10, 0, 1000), coef=B, outs=None, dt=FP, odt=None):
    zr.zr_grad_scale(at(A) if grads is None else grads, numels, coef, outs, dtype=dt, out_dtype=odt, stream=0)


def test_scale_refusals():
    expect(zr.ZR_ERR_INVALID, scale, coef=None)
    expect(zr.ZR_ERR_ALIGN, scale, coef=B + 1)
    expect(zr.ZR_ERR_ALIAS, scale, coef=A + 4)                          # inside a gradient that is written
    expect(zr.ZR_ERR_ALIAS, scale, grads=[A, B, A + 36])                # in place, two that overlap
    expect(zr.ZR_ERR_ALIAS, scale, grads=[A, C, A], numels=(8, 0, 8))   # the same twice, written
    expect(zr.ZR_ERR_ALIAS, scale, outs=[A + 4, D, E], odt=FP)          # shifted in place
    expect(zr.ZR_ERR_ALIAS, scale, outs=at(A), odt=BF)                  # in place, other type
    expect(zr.ZR_ERR_ALIAS, scale, outs=[A + 2 * GAP, D, A], odt=FP)    # another's place
    expect(zr.ZR_ERR_ALIAS, scale, outs=[D, E, D + 36], odt=FP)
    expect(zr.ZR_ERR_ALIAS, scale, outs=[D, E, B - 8], odt=FP)          # an output over coef
    expect(zr.ZR_ERR_INVALID, scale, outs=[D, E, 0], odt=FP)
    expect(zr.ZR_ERR_ALIGN, scale, outs=[D, E, F + 1], odt=BF)
    expect(zr.ZR_ERR_UNSUPPORTED, scale, outs=[D, E, F], odt=zr.ZR_CKPT_INT8)
    lib = zr.lib()
    n = (ctypes.c_int64 * 1)(5)
    assert lib.zr_grad_scale(1, zr.table([A]), n, FP, None, BF, B, None) == zr.ZR_ERR_UNSUPPORTED


def adamw(grads=None, numels=(10, 0, 1000), p=None, m=None, v=None, shards=None, step=1, coef=G, dt=BF, lr=1e-3, **kw):
    zr.zr_adamw(at(A) if grads is None else grads, numels, p or at(B), m or at(C), v or at(D), step, lr, shards=shards,
                coef=coef, dtype=dt, stream=0, **kw)


def test_adamw_refusals():
    for k in ("beta1", "beta2"):
        for bad in (-0.1, 1.0, float("nan")):
            expect(zr.ZR_ERR_INVALID, adamw, **{k: bad})
    for k in ("lr", "eps", "weight_decay"):
        for bad in (-1e-3, float("inf"), float("nan")):
            expect(zr.ZR_ERR_INVALID, adamw, **{k: bad})
    for step in (0, -5):
        expect(zr.ZR_ERR_INVALID, adamw, step=step)
    expect(zr.ZR_ERR_UNSUPPORTED, adamw, dt=9)
    for k in ("p", "m", "v"):
        expect(zr.ZR_ERR_INVALID, adamw, **{k: [E, F, 0]})
        expect(zr.ZR_ERR_ALIGN, adamw, **{k: [E, F, F + 2]})
        expect(zr.ZR_ERR_ALIAS, adamw, **{k: [E, F, A + 2 * GAP]})
        expect(zr.ZR_ERR_ALIAS, adamw, **{k: [E, F, E + 36]})
    expect(zr.ZR_ERR_ALIAS, adamw, m=at(B))
    expect(zr.ZR_ERR_ALIAS, adamw, shards=at(B))
    expect(zr.ZR_ERR_ALIAS, adamw, shards=at(A))
    expect(zr.ZR_ERR_ALIAS, adamw, coef=B + 4)
    expect(zr.ZR_ERR_ALIGN, adamw, shards=[E, F, F + 1])
    with pytest.raises(ValueError, match="entries"):
        adamw(shards=[E])
    lib = zr.lib()
    n = (ctypes.c_int64 * 1)(5)
    t = zr.table([A])
    assert lib.zr_adamw(1, t, BF, n, None, t, t, None, 1e-3, .9, .9, 1e-8, 0, 1, None, None) == zr.ZR_ERR_INVALID


def test_tensors_are_checked():
    import torch
    x = [torch.zeros(10), torch.zeros(4)]
    with pytest.raises(ValueError, match="not on the GPU"):
        zr.zr_grad_norm(x, [10, 4], B, workspace=(C, 1 << 20), stream=0)
    with pytest.raises(ValueError, match="not on the GPU"):
        zr.tensor_table(x, [10, 4])
    with pytest.raises(TypeError, match="unsupported dtype"):
        zr.zr_grad_norm([torch.zeros(3, dtype=torch.float64)], [3], B, workspace=(C, 1 << 20), stream=0)
    t = zr.tensor_table(at(A), [5, 6, 7], dtype=FP)
    with pytest.raises(ValueError, match="other sizes"):
        zr.zr_grad_norm(t, [5, 6, 8], B, workspace=(C, 1 << 20), stream=0)
    with pytest.raises(ValueError, match="dtype argument"):
        zr.zr_grad_norm(t, [5, 6, 7], B, workspace=(C, 1 << 20), dtype=BF, stream=0)


def test_workspace_of_the_longest_lists():
    """No size is formed in 32 bits on the way."""
    top = 2 ** 31 - 1
    for n in (top, top - 190, top - 191, 1 << 30):
        assert zr.zr_grad_norm_workspace_bytes(n) == -(-n // 192) * 2048 * 8


def test_adamw_counter_refusals():
    for bad in (G + 12, B + 8, A + 2 * GAP + 8, D + 2 * GAP + 3992):
        expect(zr.ZR_ERR_ALIGN if bad == G + 12 else zr.ZR_ERR_ALIAS, adamw, left_out=bad)
    expect(zr.ZR_ERR_ALIAS, adamw, left_out=G, coef=G + 4)
    expect(zr.ZR_ERR_INVALID, adamw, left_out=G + 8, step=0)
    import torch
    for bad in (torch.zeros(1), torch.zeros(2, dtype=torch.int64), torch.zeros(1, dtype=torch.float64)):
        with pytest.raises(ValueError, match="left_out is not 1"):
            adamw(left_out=bad)
