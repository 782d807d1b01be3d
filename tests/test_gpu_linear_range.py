"""Products of packed matrices at the ends of the exponents' range, every form and pair of formats.

Bounds as in test_gpu_linear; where results are below the normal range, each of the in / 8 + 48 adds loses at most half
of fp32's smallest step, 2^-150, more, and the rounding to bf16 half of its smallest, 2^-134.
"""
import numpy as np
import pytest

from test_gpu_linear import FMT, HALF, PAIRS, bound, packed, td, workspace

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("xf,wf", PAIRS)
@pytest.mark.parametrize("rows,inn,out", [(3, 300, 40), (90, 1000, 70), (300, 96, 200)])
def test_ends_of_the_range(rows, inn, out, xf, wf):
    """The smallest blocks, whose codes are subnormal, by large ones, and the reverse; results below the normal range."""
    import torch
    import gradient_sync_zr_amd as z
    for ex, ew in ((-124, 100), (110, -126), (119, -120), (-70, -70), (-66, -64)):
        rng = np.random.default_rng(inn)
        e = np.repeat(rng.integers(-3, 4, (1, -(-inn // 32))), 32, 1)[:, :inn].astype(float)
        x, w = rng.standard_normal((rows, inn)) * 2.0 ** (ex + e), rng.standard_normal((out, inn)) * 2.0 ** (ew - e)
        px, hx = packed(x, xf)
        pw, hw = packed(w, wf)
        want = hx @ hw.T   # (of e2m1 what is below 2^-126 is held as 0: a whole w may be)
        for zd in ("bf16", "fp32"):
            zt = torch.empty(rows, out, dtype=td(zd), device="cuda")
            z.zr_ckpt_linear(px, pw, rows, inn, out, zt, x_format=FMT[xf], w_format=FMT[wf], workspace=workspace(rows, inn, out))
            lim = bound(hx, hw, xf, wf, zd) + (inn / 8 + 48) * 2.0 ** -150
            lim = lim + HALF[zd] * (np.abs(want) + lim) + (2.0 ** -134 if zd == "bf16" else 2.0 ** -150)
            assert (np.abs(zt.double().cpu().numpy() - want) <= lim).all(), (ex, ew, zd)
