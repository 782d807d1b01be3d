"""The norm and checkpoint calls' argument checks under the address and
undefined-behaviour sanitizers: the C-ABI layer built without the kernels, as
for the other calls' checks."""
from test_sanitizers_cpu import builds, run_tests  # noqa: F401  (builds is a fixture)


def test_norm_and_checkpoint_calls_under_sanitizers(builds):  # noqa: F811
    run_tests(["test_norm_abi_cpu.py"], {"ZR_LIBRARY": builds["zr"]})
