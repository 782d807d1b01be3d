"""The argument checks of the gradient, RMS norm, packing and linear layer calls
under the address and undefined-behaviour sanitizers (the C-ABI layer built without
the kernels)."""
from test_sanitizers_cpu import builds, run_tests  # noqa: F401  (builds is a fixture)


def test_more_calls_under_sanitizers(builds):  # noqa: F811
    run_tests(["test_grads_abi_cpu.py", "test_rms_abi_cpu.py"], {"ZR_LIBRARY": builds["zr"]})
