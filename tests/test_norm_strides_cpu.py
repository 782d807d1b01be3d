"""Row strides of any size: refused where the rows would not fit 2^40 elements,
without arithmetic that overflows on the way (also run under the
undefined-behaviour sanitizer, which reports it where it happens)."""
import pytest

import gradient_sync_zr_amd as zr
from test_abi_cpu import A

B, C, D, E, F, G = (A + (i << 36) for i in range(1, 7))
BF, FP, E4 = zr.ZR_BF16, zr.ZR_FP32, zr.ZR_CKPT_E4M3
TOP = (1 << 63) - 1


def calls(rows, ld):
    lib = zr.lib()
    yield lib.zr_ckpt_pack(A, BF, rows, 8, ld, B, E4, None)
    yield lib.zr_ckpt_unpack(B, E4, rows, 8, A, FP, ld, None)
    yield lib.zr_layernorm_fwd(A, BF, rows, 8, ld, None, None, FP, 1e-5, B, BF, 8, None, None, None, None, E4, None)
    yield lib.zr_layernorm_fwd(A, BF, rows, 8, 8, None, None, FP, 1e-5, B, BF, ld, None, None, None, None, E4, None)
    for i in range(3):
        lds = [ld if i == k else 8 for k in range(3)]
        yield lib.zr_layernorm_bwd(A, BF, lds[0], B, BF, lds[1], rows, 8, None, FP, C, D, E, BF, lds[2], None, None, FP, 0,
                                   None, 0, None)
    yield lib.zr_ckpt_wgrad(A, BF, ld, B, E4, rows, 8, 8, C, FP, 8, None, 2, D, 1 << 30, None)


@pytest.mark.parametrize("ld", [TOP, TOP - 30, TOP - 31, TOP - 32, TOP // 2, 1 << 62, (1 << 40) + 1, 1 << 40])
def test_strides_up_to_the_largest(ld):
    for rows in (2, 1 << 39, TOP):
        assert list(calls(rows, ld)) == [zr.ZR_ERR_INVALID] * 8
    assert list(calls(0, ld)) == [zr.ZR_OK] * 8       # no rows: no extent
    if ld > 1 << 40:
        assert list(calls(1, ld)) == [zr.ZR_ERR_INVALID] * 8


def test_weight_gradient_rows():
    lib = zr.lib()
    for ld in (TOP, TOP - 31, 1 << 40):
        assert lib.zr_ckpt_wgrad(A, BF, 8, B, E4, 4, 8, 8, C, FP, ld, None, 0, D, 1 << 30, None) == zr.ZR_ERR_INVALID
