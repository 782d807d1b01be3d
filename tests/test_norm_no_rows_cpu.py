"""Calls without rows: what they add to stays as it is, so there is no work and
nothing is launched (these run without a GPU)."""
import gradient_sync_zr_amd as zr
from test_abi_cpu import A, expect

B, C, D, E, F = (A + (i << 36) for i in range(1, 6))
BF, FP = zr.ZR_BF16, zr.ZR_FP32


def test_added_gradients_stay():
    for dt in (BF, FP):
        for dw, db in ((E, F), (E, None), (None, F)):
            zr.zr_layernorm_bwd(A, B, 0, 64, C, D, dweight=dw, dbias=db, accumulate=True, dy_dtype=BF, x_dtype=BF,
                                grad_dtype=dt, stream=0)
            zr.zr_layernorm_bwd(A, B, 0, 20000, C, D, dx=A, dweight=dw, dbias=db, accumulate=True, add_dx=True,
                                dy_dtype=BF, x_dtype=BF, dx_dtype=BF, grad_dtype=dt, stream=0)
        for db in (None, F):
            zr.zr_ckpt_wgrad(A, B, 0, 40, 64, E, dbias=db, accumulate=True, dy_dtype=BF, grad_dtype=dt, stream=0)


def test_arguments_are_checked_all_the_same():
    expect(zr.ZR_ERR_ALIGN, lambda **k: zr.zr_layernorm_bwd(A, B, 0, 64, C, D, dweight=E + 2, accumulate=True,
                                                            dy_dtype=BF, x_dtype=BF, grad_dtype=FP, stream=0))
    expect(zr.ZR_ERR_ALIAS, lambda **k: zr.zr_ckpt_wgrad(A, B, 0, 40, 64, E, dbias=E + 4, accumulate=True, dy_dtype=BF,
                                                         grad_dtype=FP, stream=0))


def test_outputs_without_rows_have_no_address():
    """An empty tensor's address is 0, which is an output's that is not given, too: without rows both are no work."""
    lib = zr.lib()
    for x_dt in (BF, zr.ZR_CKPT_E4M3):
        assert lib.zr_layernorm_fwd(None, x_dt, 0, 64, 64, E, F, BF, 1e-5, None, BF, 64, None, None, None, None, BF,
                                    None) == zr.ZR_OK
        assert lib.zr_layernorm_bwd(None, BF, 64, None, x_dt, 64, 0, 64, E, BF, None, None, None, BF, 64, None, None, FP, 0,
                                    None, 0, None) == zr.ZR_OK
    assert lib.zr_ckpt_pack(None, BF, 0, 64, 64, None, zr.ZR_CKPT_INT8, None) == zr.ZR_OK
    assert lib.zr_ckpt_unpack(None, zr.ZR_CKPT_INT8, 0, 64, None, BF, 64, None) == zr.ZR_OK
    # with rows an output is needed
    assert lib.zr_layernorm_fwd(A, BF, 1, 64, 64, E, F, BF, 1e-5, None, BF, 64, None, None, None, None, BF,
                                None) == zr.ZR_ERR_INVALID
