"""RMS norm at the ends of its values: backward with a NaN or an infinity in any operand, in every form of the
kernels, and forward of rows whose squares pass fp32."""
import pytest

from test_gpu_norm import code

pytestmark = pytest.mark.gpu

# 16 and 64 lanes a row, 256 and 512 with one to three vectors each, and the wide form; borders between them
COLS = [24, 300, 1000, 2048, 4095, 8192, 12001, 13001]


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("hd", ["bf16", "fp32", "e4m3", "int8"])
def test_backward_of_values_that_are_not_finite(hd, cols):
    """A bad value leaves nothing finite of its row of dx and of its column of dweight (of its block's where h is a
    checkpoint, of all columns where it is rstd), and every other element's bits as they were."""
    import torch
    import gradient_sync_zr_amd as z
    rows, r, j = 9, 4, cols // 2
    g = torch.Generator("cuda").manual_seed(cols)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    h, dy = rand(rows, cols).bfloat16(), rand(rows, cols).bfloat16()
    h[r, j], dy[r, j] = 0.5, 0.5   # an infinity of the other one does not meet a zero
    w, rstd = rand(cols).abs() + 0.5, torch.rand(rows, generator=g, device="cuda") + 0.5
    ws = torch.empty(max(1, z.zr_rmsnorm_workspace_bytes(rows, cols)), dtype=torch.uint8, device="cuda")

    def run(h, dy, rstd):
        if hd in ("e4m3", "int8"):
            src = torch.empty(z.zr_ckpt_bytes(rows, cols), dtype=torch.uint8, device="cuda")
            z.zr_ckpt_pack(h, rows, cols, src, format=code(hd))
        else:
            src = h if hd == "bf16" else h.float()
        dx, dw = torch.empty(rows, cols, device="cuda"), torch.empty(cols, device="cuda")
        z.zr_rmsnorm_bwd(dy, src, rows, cols, rstd, w, dx=dx, dweight=dw, workspace=ws,
                         h_dtype=code(hd) if hd in ("e4m3", "int8") else None)
        return dx, dw

    dx0, dw0 = run(h, dy, rstd)
    assert bool(torch.isfinite(dx0).all()) and bool(torch.isfinite(dw0).all())
    other = torch.arange(rows, device="cuda") != r
    for where in ("h", "dy", "rstd"):
        for bad in (float("nan"), float("inf"), float("-inf")) if where != "rstd" else (float("nan"),):
            a, b, c = h.clone(), dy.clone(), rstd.clone()
            hit = torch.zeros(cols, dtype=torch.bool, device="cuda")
            if where == "h":
                a[r, j] = bad
                hit[j] = True
                if hd in ("e4m3", "int8"):
                    hit[j // 32 * 32:j // 32 * 32 + 32] = True
            elif where == "dy":
                b[r, j] = bad
                hit[j] = True
            else:
                c[r] = bad
                hit[:] = True
            dx, dw = run(a, b, c)
            assert not bool(torch.isfinite(dx[r]).any()), (where, bad)
            assert torch.equal(dx[other], dx0[other]), (where, bad)
            assert not bool(torch.isfinite(dw[hit]).any()) and torch.equal(dw[~hit], dw0[~hit]), (where, bad)


@pytest.mark.parametrize("cols", [24, 300, 4096, 17000])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_forward_of_rows_whose_squares_pass_fp32(dt, cols):
    """2^64 squared is beyond fp32: rstd and y of the row are 0, in 64 bits they would be 2^-64 and 1. Just below, rows
    are normed; rows beside them do not change."""
    import torch
    import gradient_sync_zr_amd as z
    x = torch.randn(4, cols, device="cuda").to(torch.bfloat16 if dt == "bf16" else torch.float32)
    y, rstd, y0, rstd0 = torch.empty_like(x), torch.empty(4, device="cuda"), torch.empty_like(x), torch.empty(4, device="cuda")
    z.zr_rmsnorm_fwd(x, 4, cols, y0, rstd=rstd0)
    x[1] = 2.0 ** 64
    x[2] = 2.0 ** 56   # its squares' sum, up to 17000 * 2^112, is below 2^127
    z.zr_rmsnorm_fwd(x, 4, cols, y, rstd=rstd)
    assert float(rstd[1]) == 0.0 and bool((y[1] == 0).all())
    assert float(rstd[2]) == 2.0 ** -56 and bool((y[2] == 1).all())
    assert torch.equal(y[[0, 3]], y0[[0, 3]]) and torch.equal(rstd[[0, 3]], rstd0[[0, 3]])
