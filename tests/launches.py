"""What the library's calls would launch, without a GPU: a child process loads
tests/kit/launch_log.cpp in front of the library, makes the calls with addresses
that nothing reads, and reports each call's kernels, blocks and threads."""
import json
import os
import re
import subprocess
import sys

from conftest import ROOT

KIT = os.path.join(ROOT, "tests", "kit")
LOG = os.path.join(KIT, "liblaunch_log.so")

CHILD = """
import ctypes, json, sys
sys.path.insert(0, sys.argv[1])
log = ctypes.CDLL(sys.argv[2], mode=ctypes.RTLD_GLOBAL)   # before the library: its symbols are found first
log.ll_launch.restype = ctypes.c_char_p
import gradient_sync_zr_amd as zr
lib = zr.lib()
out = []
for name, args in json.load(sys.stdin):
    log.ll_clear()
    status = getattr(lib, name)(*args)
    got = []
    for i in range(log.ll_count()):
        dims = (ctypes.c_uint32 * 6)()
        got.append([log.ll_launch(i, dims).decode(), list(dims)])
    out.append([status, got, zr.zr_last_error() if status else ""])
print(json.dumps(out))
"""


def launches(calls, env=None):
    """Of each call (name, arguments): [(kernel's name, blocks, threads per block), ...]."""
    if not os.path.exists(LOG):
        sys.path.insert(0, os.path.join(ROOT, "tests"))
        from kit import _build
        _build.build()
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT, LOG], input=json.dumps(calls), capture_output=True, text=True,
                       env=dict(os.environ, **(env or {})), timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    out = []
    for status, got, error in json.loads(r.stdout):
        assert status == 0, error
        out.append([])
        for symbol, d in got:
            assert d[1] == d[2] == d[4] == d[5] == 1
            name = max(re.findall(r"\d+([a-z_0-9]+kernel)", symbol), key=len)   # of a mangled symbol
            out[-1].append((name, d[0], d[3]))
    return out
