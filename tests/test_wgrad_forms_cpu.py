"""Which form of the weight gradient the sizes of the GPU tests take: what a
launch of the real library would be, without a GPU."""
import ckpt_ref as ref
import gradient_sync_zr_amd as zr
import test_gpu_ckpt
import test_gpu_wgrad_large as big
from launches import launches
from test_launch_sizes_cpu import wgrad

BF, FP = zr.ZR_BF16, zr.ZR_FP32


def kernels(sizes, dy_dt=BF):
    return [[k for k, _, _ in got] for got in launches([wgrad(*s, dy_dt) for s in sizes])]


def test_large_form():
    for s, got in zip(big.WHOLE, kernels(big.WHOLE)):
        assert got == ["wgrad_big_kernel"], s
    split = big.SPLIT + [big.FAR]
    for s, got in zip(split, kernels(split)):
        assert got == ["wgrad_big_kernel", "wgrad_big_join_kernel"], s
    sizes = [big.EXPONENTS] + [(4000, 4300, 4100), (200000, 40, 70), (700, 4097, 4100)]
    for s, got in zip(sizes, kernels(sizes)):
        assert got[0] == "wgrad_big_kernel", s


def test_small_form():
    """bf16 dy at the sizes of the small form's tests, and fp32 dy at every size."""
    sizes = test_gpu_ckpt.WSHAPES + [big.SMALL_EXPONENTS, (600, 264, 300), (1100, 130, 33)]
    for s, got in zip(sizes, kernels(sizes)):
        assert got[0] == "wgrad_kernel", s
    sizes += big.WHOLE + big.SPLIT
    for s, got in zip(sizes, kernels(sizes, FP)):
        assert got[0] == "wgrad_kernel", s


def test_dy_that_the_large_form_cannot_read():
    """Less than a chunk of 8 columns, or rows whose offsets within a slab pass 32 bits."""
    far = [(200000, 7, 70)]
    assert kernels(far)[0][0] == "wgrad_kernel"
    name, args = wgrad(700, 4104, 4100)
    args[2] = (1 << 24) + 1
    assert launches([(name, args)])[0][0][0] == "wgrad_kernel"
    args[2] = 1 << 24
    assert launches([(name, args)])[0][0][0] == "wgrad_big_kernel"


def test_both_forms_and_joins_are_reached():
    got = kernels([(700, 4104, 4100), (4000, 4300, 4100), (64, 129, 127), (8192, 100, 70)])
    assert got == [["wgrad_big_kernel"], ["wgrad_big_kernel", "wgrad_big_join_kernel"], ["wgrad_kernel"],
                   ["wgrad_kernel", "wgrad_join_kernel"]]
    assert ref.E4M3 == zr.ZR_CKPT_E4M3
