"""HIP refuses a launch of 2^32 work-items or more. The norm, checkpoint and
weight gradient calls take sizes at which one block per tile or row would be
more: their launches stay below it, and the blocks stride over the rest."""
import pytest

import gradient_sync_zr_amd as zr
from launches import launches
from test_abi_cpu import A

BF, FP = zr.ZR_BF16, zr.ZR_FP32
E4, I8 = zr.ZR_CKPT_E4M3, zr.ZR_CKPT_INT8
FAR = 1 << 44    # further apart than any buffer is long
B, C, D, E, F, G, H = (FAR * (i + 8) for i in range(1, 8))


def fwd(rows, cols, x_dt=BF):
    ld = cols
    return "zr_layernorm_fwd", [B, x_dt, rows, cols, ld, None, None, FP, 1e-5, C, BF, ld, D, E, None, None, E4, None]


def bwd(rows, cols, dx=True, grads=True, x_dt=BF, dy_dt=BF):
    return "zr_layernorm_bwd", [B, dy_dt, cols, C, x_dt, cols, rows, cols, None, FP, D, D + FAR // 2, E if dx else None, BF,
                                cols, F if grads else None, F + FAR // 2 if grads else None, FP, 0, G, FAR, None]


def wgrad(rows, out, inn, dy_dt=BF, fmt=E4):
    return "zr_ckpt_wgrad", [B, dy_dt, out, C, fmt, rows, out, inn, D, BF, inn, E, 0, G, FAR, None]


CALLS = {
    "wide rows forward": fwd((1 << 22) + 3, 16385),
    "wide rows forward, from a checkpoint": fwd((1 << 22) + 3, 16385, I8),
    "narrow rows forward": fwd(1 << 32, 64),
    "wide rows backward": bwd((1 << 22) + 3, 12289, grads=False),
    "wide rows backward, from a checkpoint": bwd(1 << 23, 12289, x_dt=E4, dy_dt=FP),
    "wide column sums": bwd(300, 1 << 27, dx=False),
    "join of one row": bwd(1, 1 << 27),
    "join of the widest rows": bwd(1 << 10, 1 << 30),
    "narrow rows backward": bwd(1 << 33, 100),
    "pack": ("zr_ckpt_pack", [B, BF, 1 << 20, 1 << 20, 1 << 20, C, E4, None]),
    "unpack": ("zr_ckpt_unpack", [B, I8, 1 << 20, 1 << 20, C, FP, 1 << 20, None]),
    "weight gradient, many tiles": wgrad(1, 1 << 20, 1 << 20),
    "weight gradient, long and narrow": wgrad(100, 1 << 30, 1000),
    "weight gradient, fp32": wgrad(100, 1 << 30, 1000, FP),
    "weight gradient, many rows": wgrad(1 << 33, 128, 128),
}


def test_launches_stay_below_the_limit():
    for name, got in zip(CALLS, launches(list(CALLS.values()))):
        assert got, name
        for kernel, blocks, threads in got:
            assert 0 < blocks and blocks * threads < 1 << 32, (name, kernel, blocks, threads)


def test_small_launches_have_a_block_per_item():
    """The cap leaves launches below it as they are."""
    got = launches([fwd(1000, 20000), bwd(7, 13000), ("zr_ckpt_pack", [B, BF, 1 << 10, 1 << 10, 1 << 10, C, E4, None])])
    assert got[0] == [("fwd_wide_kernel", 1000, 1024)]
    assert got[1] == [("bwd_wide_sums_kernel", 7 * 7, 256), ("bwd_wide_dx_kernel", 7, 1024), ("bwd_join_kernel", 407, 1024)]
    assert got[2] == [("pack_kernel", 128, 256)]


@pytest.mark.parametrize("cap", ["13", "1"])
def test_launches_keep_to_a_lowered_cap(cap):
    for name, got in zip(CALLS, launches(list(CALLS.values()), {"ZR_MAX_GRID": cap})):
        for kernel, blocks, _ in got:
            assert 0 < blocks <= int(cap), (name, kernel, blocks)
