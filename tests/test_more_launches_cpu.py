"""Which kernels the gradient, RMS norm, packing and linear layer calls launch, and
in how many blocks, from the library's launches with the runtime's entry points
replaced (no GPU)."""
import json
import subprocess
import sys

import gradient_sync_zr_amd as zr
from conftest import ROOT
from launches import LOG, launches

BF, FP, E4, E2 = zr.ZR_BF16, zr.ZR_FP32, zr.ZR_CKPT_E4M3, zr.ZR_CKPT_E2M1
FAR = 1 << 44


def test_launches_stay_below_the_limit():
    """HIP refuses 2^32 work-items; sizes that would be more in one block per tile or row stride over the rest."""
    b, c, d, e, f, g = (FAR * (i + 8) for i in range(1, 7))
    lin = lambda rows, inn, out: ("zr_ckpt_linear", [b, E4, c, E2, rows, inn, out, None, BF, d, BF, out, 0, e, FAR, None])  # noqa: E731
    calls = {
        "wide rows forward": ("zr_rmsnorm_fwd", [b, BF, (1 << 22) + 3, 16385, 16385, None, 16385, None, 16385, BF, None, FP,
                                                 1e-5, c, BF, 16385, d, None, None, E4, None]),
        "narrow rows forward": ("zr_rmsnorm_fwd", [b, BF, 1 << 32, 64, 64, c, 64, d, 64, BF, None, FP, 1e-5, e, BF, 64, f, None,
                                                   None, E4, None]),
        "wide rows backward": ("zr_rmsnorm_bwd", [b, BF, 12289, c, BF, 12289, (1 << 22) + 3, 12289, None, FP, d, e, BF, 12289,
                                                  None, FP, 0, g, FAR, None]),
        "column sums": ("zr_rmsnorm_bwd", [b, BF, 1 << 27, c, E4, 1 << 27, 300, 1 << 27, None, FP, d, None, BF, 1 << 27, f, FP,
                                           0, g, FAR, None]),
        "join of the widest rows": ("zr_rmsnorm_bwd", [b, BF, 1 << 30, c, BF, 1 << 30, 1 << 10, 1 << 30, None, FP, d, None, BF,
                                                       1 << 30, f, FP, 0, g, FAR, None]),
        "pack": ("zr_ckpt_pack", [b, BF, 1 << 20, 1 << 20, 1 << 20, c, E2, None]),
        "unpack": ("zr_ckpt_unpack", [b, E2, 1 << 20, 1 << 20, c, FP, 1 << 20, None]),
        "transposed pack": ("zr_ckpt_pack_t", [b, BF, 1 << 20, 1 << 20, 1 << 20, c, E4, None]),
        "transposed pack of few rows": ("zr_ckpt_pack_t", [b, BF, 40, 1 << 30, 1 << 30, c, E2, None]),
        "many tiles": lin(1 << 20, 32, 1 << 20),
        "many tokens": lin(1 << 33, 128, 128),
        "many outputs": lin(100, 1000, 1 << 30),
        "few tokens": lin(3, 1000, 1 << 30),
        "wide operands": lin(1 << 10, 1 << 30, 1 << 10),
    }
    for env in (None, {"ZR_MAX_GRID": "13"}):
        for name, got in zip(calls, launches(list(calls.values()), env)):
            assert got, name
            for kernel, blocks, threads in got:
                assert 0 < blocks <= (13 if env else 1 << 30) and blocks * threads < 1 << 32, (name, kernel, blocks, threads)


def test_forms_of_the_product():
    """Few rows, tiles of 128 and of 256, and columns in parts with a join, as the time model has them."""
    b, c, d, e = (FAR * (i + 8) for i in range(1, 5))
    lin = lambda rows, inn, out, x=E4, w=E4, z=BF: ("zr_ckpt_linear", [b, x, c, w, rows, inn, out, None, BF, d, z, out, 0, e,  # noqa: E731
                                                                        FAR, None])
    few, tiles, join = "linear_few_kernel", "linear_kernel", "linear_join_kernel"
    got = launches([lin(1, 4096, 4096), lin(64, 1000, 777), lin(64, 4096, 11008), lin(1024, 1024, 1024), lin(4096, 4096, 4096),
                    lin(128, 4096, 4096), lin(16384, 4096, 11008, E2, E2)])
    assert got[0] == [(few, 256, 512)] and got[1] == [(few, 49, 512)]
    assert got[2][0][0] == tiles
    assert got[3] == [(tiles, 64, 256)] and got[4] == [(tiles, 256, 512)]
    assert got[5][0] == (tiles, 128, 256) and got[5][1][0] == join
    assert [k for k, _, _ in got[6]] == [tiles]
    assert zr.zr_ckpt_linear_workspace_bytes(128, 4096, 4096) == 4 * 4 * 128 * 4096
    # 256 x 256 for a tall product in every kind (129 tiles), and in 7 parts
    got = launches([lin(32847, 600, 131, E4, E4, BF), lin(32847, 600, 131, E2, E2, BF), lin(32847, 600, 131, E4, E4, FP),
                    lin(32847, 600, 131, E2, E2, FP), lin(8662, 13958, 130)])
    assert [g[0] for g in got] == [(tiles, 129, 512)] * 4 + [(tiles, 238, 512)] and got[4][1][0] == join


def test_launches():
    """One block up to 16384 elements in four tiles; a block per tile and a join beyond; a launch per 192, 128 or 64 tensors."""
    launches([])  # builds the library that writes launches down
    code = """
import ctypes, json, sys
sys.path.insert(0, sys.argv[1])
log = ctypes.CDLL(sys.argv[2], mode=ctypes.RTLD_GLOBAL)
log.ll_launch.restype = ctypes.c_char_p
import gradient_sync_zr_amd as zr
A = 1 << 46
out = []
for what, n, numel in json.loads(sys.argv[3]):
    log.ll_clear()
    t = [A + i * (1 << 35) for i in range(n)]
    far = lambda k: [x + (k << 43) for x in t]
    if what == "norm":
        zr.zr_grad_norm(t, [numel] * n, 4096, 8192, workspace=(1 << 20, 1 << 30), dtype=1, stream=0)
    elif what == "scale":
        zr.zr_grad_scale(t, [numel] * n, 4096, dtype=1, stream=0)
    else:
        zr.zr_adamw(t, [numel] * n, far(1), far(2), far(3), 1, 1e-3, shards=far(4), coef=4096, dtype=1, stream=0)
    got = []
    for i in range(log.ll_count()):
        d = (ctypes.c_uint32 * 6)()
        got.append([log.ll_launch(i, d).decode(), d[0], d[3]])
    out.append(got)
print(json.dumps(out))
"""
    asked = [["norm", 0, 0], ["norm", 5, 0], ["norm", 1, 16384], ["norm", 4, 4000], ["norm", 5, 4000], ["norm", 1, 1 << 34],
             ["norm", 193, 5000], ["scale", 1, 4097], ["scale", 128, 10], ["scale", 129, 10], ["scale", 3, 0],
             ["adamw", 64, 4096], ["adamw", 130, 4097], ["adamw", 1, 1 << 34]]
    r = subprocess.run([sys.executable, "-c", code, ROOT, LOG, json.dumps(asked)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    got = json.loads(r.stdout)
    name = lambda s: next(k for k in ("norm_one", "norm_join", "norm_kernel", "scale_kernel", "adamw_kernel") if k in s)  # noqa: E731
    got = [[(name(s), b, t) for s, b, t in g] for g in got]
    one, join = ("norm_one", 1, 1024), ("norm_join", 1, 1024)
    # (tiles of the norm have 8192 elements, of the others 4096)
    assert got[:4] == [[one]] * 4
    assert got[4] == [("norm_kernel", 5, 256), join]
    assert got[5] == [("norm_kernel", 2048, 256), join]
    assert got[6] == [("norm_kernel", 192, 256), ("norm_kernel", 1, 256), join]
    assert got[7] == [("scale_kernel", 2, 256)] and got[8] == [("scale_kernel", 128, 256)]
    assert got[9] == [("scale_kernel", 128, 256), ("scale_kernel", 1, 256)] and got[10] == []
    assert got[11] == [("adamw_kernel", 64, 256)]
    assert got[12] == [("adamw_kernel", 128, 256)] * 2 + [("adamw_kernel", 4, 256)]
    assert len(got[13]) == 1 and all(b * t < 1 << 32 for g in got for _, b, t in g)


def test_forms_of_up_to_64_rows():
    """The border between the form of few rows and tiles, at sizes where one was measured to take a third less and more."""
    b, c, d, e = (FAR * (i + 8) for i in range(1, 5))
    lin = lambda rows, inn, out, x, w, z=BF: ("zr_ckpt_linear", [b, x, c, w, rows, inn, out, None, BF, d, z, out, 0, e, FAR, None])  # noqa: E731
    few = [lin(17, 11008, 4096, E2, E2), lin(24, 11008, 4096, E2, E2), lin(33, 4096, 4096, E2, E2), lin(17, 4096, 512, E4, E4),
           lin(8, 8192, 1024, E4, E4, FP), lin(24, 8192, 1024, E2, E2, FP), lin(17, 1000, 777, E4, E4), lin(40, 2560, 640, E4, E4, FP),
           lin(1, 16384, 8192, E4, E2)]
    tiles = [lin(64, 4096, 11008, E4, E4), lin(64, 4096, 11008, E2, E2), lin(8, 1024, 32768, E2, E2), lin(64, 16384, 8192, E4, E4),
             lin(64, 2048, 16384, E4, E4), lin(33, 1024, 32768, E4, E4, FP)]
    assert [k[0][0] for k in launches(few)] == ["linear_few_kernel"] * len(few)
    assert [k[0][0] for k in launches(tiles)] == ["linear_kernel"] * len(tiles)
