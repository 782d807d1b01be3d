"""More of the norm and checkpoint calls' argument checks under the address and
undefined-behaviour sanitizers (the C-ABI layer built without the kernels)."""
from test_sanitizers_cpu import builds, run_tests  # noqa: F401  (builds is a fixture)


def test_norm_calls_under_sanitizers(builds):  # noqa: F811
    run_tests(["test_norm_strides_cpu.py", "test_norm_dtypes_cpu.py", "test_norm_no_rows_cpu.py"],
              {"ZR_LIBRARY": builds["zr"]})
