"""The norm, checkpoint and weight gradient kernels with their grids capped at
13 blocks (ZR_MAX_GRID, read once when the library loads, so a child process of
its own): the loops over rows, tiles and parts that a full grid enters at
very large sizes alone."""
import os
import subprocess
import sys

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("module,which", [
    ("test_gpu_ckpt.py", "not past_32"),
    ("test_gpu_norm.py", "test_forward or differences or in_place_apart"),
    ("test_gpu_norm_rows.py", "over_many_rows"),
    ("test_gpu_wgrad_large.py", "not past_32 and not test_values"),
])
def test_with_blocks_striding(module, which):
    env = dict(os.environ, ZR_MAX_GRID="13")
    cmd = [sys.executable, "-u", "-m", "pytest", os.path.join(ROOT, "tests", module), "-x", "-q", "-m", "gpu", "-k", which,
           "-p", "no:cacheprovider", "--timeout", "300", "--timeout-method", "thread"]
    print(f"strided grid: {module} with ZR_MAX_GRID=13", flush=True)
    r = subprocess.run(cmd, env=env, cwd=ROOT, capture_output=True, text=True, timeout=900)
    tail = r.stdout[-2500:] + r.stderr[-1500:]
    print(tail, flush=True)
    assert r.returncode == 0, tail
    assert " passed" in r.stdout and "failed" not in r.stdout
