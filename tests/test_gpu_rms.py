"""RMS norm on the GPU against its formulas in 64 bits.

Bounds, with u = 2^-24 and every sum of a row made of at most 64 adds in line (as in
the layer norm's tests):
 * h: one fp32 add and one rounding to its type: compared bit for bit with the same two;
 * rstd: the sum of squares is 66 u of itself, its mean 1 u more, the root half of
   both and 3 u: 37 u;
 * y: 37 u of rstd, and two products: 39 u |y|, and half a step of y's type;
 * dx: xh and g are 1 u each, the sum of g xh 66 u of its magnitudes, its factor 3 u, the
   last steps 3 u: 2 u |g| rstd + 74 u |xh| rstd mean|g xh| + 2 u of the result, with the
   added dx one more, and half a step of its type;
 * dweight: xh 1 u, and column_adds() u of the sum of magnitudes; half a step.
"""
import numpy as np
import pytest

import ckpt_ref as ref
from gpu_util import Guarded
from test_gpu_ckpt import tensor
from test_gpu_grads import bf16
from test_gpu_norm import COLS, HALF, U, code, column_adds, make, rows_of, take, td, vec

pytestmark = pytest.mark.gpu


def zr():
    import gradient_sync_zr_amd as m
    return m


def source(x, xd, cols, gap, shift):
    """(what to pass as x, its 64-bit values, what keeps it alive)."""
    import torch
    if xd in ("e4m3", "int8"):
        buf = torch.from_numpy(ref.buffer(*ref.pack(x.astype(np.float64), code(xd)))).cuda()
        return buf, ref.held(x.astype(np.float64), code(xd)), buf
    g = tensor(x, xd, cols + gap, shift)
    return g.ptr(), x.astype(np.float64), g


def strided(rows, cols, ld, dt, shift, value=3.0):
    g = Guarded((rows - 1) * ld + cols, td(dt), shift)
    g.t.fill_(value)
    return g


CASES = [(1, "bf16", "bf16", "bf16", "bf16"), (37, "fp32", "bf16", "fp32", None), (5, "bf16", "fp32", "fp32", "fp32"),
         (18, "fp32", "fp32", "bf16", "bf16"), (3, "e4m3", "bf16", "bf16", None), (33, "int8", "fp32", "fp32", "fp32"),
         (7, "e4m3", "bf16", "bf16", "bf16")]


@pytest.mark.parametrize("cols", COLS)
def test_forward(cols):
    import torch
    z = zr()
    rng = np.random.default_rng(cols)
    for k, (rows, xd, yd, pd, hd) in enumerate(CASES):
        x = make(rng, rows, cols, "bf16" if xd != "fp32" else xd)
        w = make(rng, 1, cols, pd)[0]
        weight = k != 3
        gap, shift = (5, 1) if k % 2 else (0, 0)
        ld = cols + gap
        src, x64, keep = source(x, xd, cols, gap, shift)
        gw = vec(w, pd, shift)
        gy, gr = strided(rows, cols, ld, yd, shift), Guarded(rows, torch.float32, shift)
        gh = strided(rows, cols, ld, hd, shift, 4.0) if hd else None
        r = make(rng, rows, cols, hd) if hd else None
        gres = tensor(r, hd, ld, 1 - shift) if hd else None
        cy, ch = (torch.full((ref.nbytes(rows, cols),), 0x55, dtype=torch.uint8, device="cuda") for _ in range(2))
        keeps = hd is not None or xd not in ("e4m3", "int8")
        fmt = (ref.E4M3, ref.INT8)[k % 2]
        eps = 1e-5
        z.zr_rmsnorm_fwd(src, rows, cols, gy.ptr(), gw.ptr() if weight else None, eps=eps, residual=gres.ptr() if hd else None,
                         h=gh.ptr() if hd else None, rstd=gr.ptr(), ckpt_h=ch if keeps else None, ckpt_y=cy, ckpt_format=fmt,
                         x_dtype=code(xd), y_dtype=code(yd), h_dtype=code(hd) if hd else None, param_dtype=code(pd),
                         ld_x=ld, ld_y=ld, ld_h=ld, ld_residual=ld)
        h = x64
        if hd:  # one fp32 add, one rounding
            h = x64.astype(np.float32) + r.astype(np.float32)
            h = (bf16(h) if hd == "bf16" else h).astype(np.float64)
            assert np.array_equal(rows_of(gh, hd, rows, cols, ld, 4.0), h) and gh.guards_intact()
        w64 = w.astype(np.float64) if weight else np.ones(cols)
        rstd = 1 / np.sqrt((h * h).mean(1) + eps)
        y = h * rstd[:, None] * w64
        got = rows_of(gy, yd, rows, cols, ld, 3.0)
        assert (np.abs(take(gr, "fp32") - rstd) <= 37 * U * rstd).all()
        by = 40 * U * np.abs(y)
        assert (np.abs(got - y) <= by + HALF[yd] * (np.abs(y) + by)).all()
        assert gy.guards_intact() and gr.guards_intact()
        # the checkpoints: of h, and of y as it was written, exactly
        if keeps:
            assert np.array_equal(ch.cpu().numpy(), ref.buffer(*ref.pack(h, fmt)))
        assert np.array_equal(cy.cpu().numpy(), ref.buffer(*ref.pack(got, fmt)))


def test_forward_several_turns():
    """More rows than the grid has at once, in every form: row by row what few rows give."""
    import torch
    z = zr()
    for rows, cols in ((70000, 96), (9001, 512), (9000, 1000), (2100, 2048), (2101, 4090), (1100, 8192), (1025, 12001), (1030, 16000),
                       (3, 20000)):
        g = torch.Generator("cuda").manual_seed(cols)
        x = torch.randn(rows, cols, generator=g, device="cuda").bfloat16()
        r = torch.randn(rows, cols, generator=g, device="cuda").bfloat16()
        w = torch.randn(cols, generator=g, device="cuda")
        y, h, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device="cuda")
        z.zr_rmsnorm_fwd(x, rows, cols, y, w, residual=r, h=h, rstd=rstd)
        assert torch.equal(h, x + r)
        h64 = h.double()
        want = 1 / torch.sqrt((h64 * h64).mean(1) + 1e-5)
        assert bool(((rstd.double() - want).abs() <= 37 * U * want).all())
        y64 = h64 * want[:, None] * w.double()
        assert bool(((y.double() - y64).abs() <= (2.0 ** -8 * (1 + 40 * U) + 40 * U) * y64.abs()).all())


def test_forward_in_place_and_outputs_apart():
    import torch
    z = zr()
    for cols in (100, 4095, 4096, 17001):
        x, r = (torch.randn(19, cols, device="cuda").bfloat16() for _ in range(2))
        y, h = torch.empty_like(x), torch.empty_like(x)
        z.zr_rmsnorm_fwd(x, 19, cols, y, residual=r, h=h)
        s = torch.empty(19, device="cuda")
        z.zr_rmsnorm_fwd(x, 19, cols, residual=r, rstd=s)          # the statistics alone, of the rounded sum
        for places in ("h at the residual", "h at x, y at the residual", "y at x"):
            a, b = x.clone(), r.clone()
            if places == "h at the residual":
                out, mid = torch.empty_like(x), b
            elif places == "h at x, y at the residual":
                out, mid = b, a
            else:
                out, mid = a, torch.empty_like(x)
            z.zr_rmsnorm_fwd(a, 19, cols, out, residual=b, h=mid)
            assert torch.equal(out, y) and torch.equal(mid, h), places
        ck, cw = (torch.empty(z.zr_ckpt_bytes(19, cols), dtype=torch.uint8, device="cuda") for _ in range(2))
        z.zr_rmsnorm_fwd(x, 19, cols, residual=r, ckpt_y=ck)       # h and y not written: rounded all the same
        z.zr_ckpt_pack(y, 19, cols, cw)
        assert torch.equal(ck, cw)
        plain = torch.empty_like(x)
        z.zr_rmsnorm_fwd(h, 19, cols, plain)                       # without a residual
        assert torch.equal(plain, y)
        z.zr_rmsnorm_fwd(h, 19, cols, h)
        assert torch.equal(h, y)
        both = torch.randn(19, cols, device="cuda").bfloat16()     # x is the residual
        z.zr_rmsnorm_fwd(both, 19, cols, y, residual=both, h=h)
        assert torch.equal(h, both * 2)


def test_forward_zero_rows_and_values_that_are_not_finite():
    """A row of zeros has rstd = eps^-1/2 and y = 0; a NaN makes its row NaN; other rows do not change."""
    import torch
    z = zr()
    for cols in (24, 300, 4096, 17000):
        x = torch.randn(4, cols, device="cuda")
        x[0] = 0
        x[2, cols // 2] = float("nan")
        y, rstd = torch.empty_like(x), torch.empty(4, device="cuda")
        z.zr_rmsnorm_fwd(x, 4, cols, y, rstd=rstd, eps=1e-4)
        assert bool((y[0] == 0).all()) and abs(float(rstd[0]) - 100) <= 100 * 4 * U
        assert bool(torch.isnan(y[2]).all()) and bool(torch.isfinite(y[[1, 3]]).all())
        x[2, cols // 2] = float("inf")
        z.zr_rmsnorm_fwd(x, 4, cols, y, rstd=rstd, eps=1e-4)
        # the norm of an infinite row is infinite: 0 everywhere, and not a number where the infinity is
        assert float(rstd[2]) == 0 and bool(torch.isnan(y[2, cols // 2])) and int((y[2] != 0).sum()) == 1


# --------------------------------------------------------------- backward
def backward64(dy, h, rstd, w):
    xh = h * rstd[:, None]
    g = dy * w
    c = (g * xh).mean(1, keepdims=True)
    dx = rstd[:, None] * (g - xh * c)
    bdx = rstd[:, None] * U * (2 * np.abs(g) + 74 * np.abs(xh) * np.abs(g * xh).mean(1, keepdims=True)) + 2 * U * np.abs(dx)
    return dx, (dy * xh).sum(0), bdx, np.abs(dy * xh).sum(0)


BWD = [(1, "bf16", "bf16", "bf16", "bf16", "fp32"), (37, "fp32", "bf16", "fp32", "fp32", "bf16"),
       (300, "bf16", "fp32", "fp32", "bf16", "fp32"), (3, "e4m3", "bf16", "bf16", "bf16", "bf16"),
       (70, "int8", "fp32", "fp32", "bf16", "fp32"), (18, "fp32", "fp32", "bf16", "fp32", "fp32")]


@pytest.mark.parametrize("cols", COLS)
def test_backward(cols):
    import torch
    z = zr()
    rng = np.random.default_rng(cols + 1)
    for k, (rows, hd, dd, pd, xd, gd) in enumerate(BWD):
        x = make(rng, rows, cols, "bf16" if hd != "fp32" else hd)
        w, dy = make(rng, 1, cols, pd)[0], make(rng, rows, cols, dd, 0.01)
        old, oldw = make(rng, rows, cols, xd, 0.01), make(rng, 1, cols, gd)[0]
        gap, shift = (5, 1) if k % 2 else (0, 0)
        ld = cols + gap
        src, h64, keep = source(x, hd, cols, gap, shift)
        rstd = (1 / np.sqrt((h64 * h64).mean(1) + 1e-5)).astype(np.float32)
        gr = vec(rstd, "fp32")
        gdy, gw = tensor(dy, dd, ld, shift), vec(w, pd, shift)
        add, accumulate, weight = k % 2 == 0, k in (1, 4), k != 2
        gdx = tensor(old, xd, ld, 1 - shift)
        gdw = vec(oldw, gd, shift)
        ws = torch.full((z.zr_rmsnorm_workspace_bytes(rows, cols),), 0x7F, dtype=torch.uint8, device="cuda")
        z.zr_rmsnorm_bwd(gdy.ptr(), src, rows, cols, gr.ptr(), gw.ptr() if weight else None, dx=gdx.ptr(), dweight=gdw.ptr(),
                         accumulate=accumulate, add_dx=add, workspace=ws, dy_dtype=code(dd), h_dtype=code(hd),
                         dx_dtype=code(xd), param_dtype=code(pd), grad_dtype=code(gd), ld_dy=ld, ld_h=ld, ld_dx=ld)
        dx, dw, bdx, magw = backward64(dy.astype(np.float64), h64, rstd.astype(np.float64),
                                       w.astype(np.float64) if weight else np.ones(cols))
        if add:
            dx = dx + old.astype(np.float64)
            bdx = bdx + 2 * U * (np.abs(dx) + np.abs(old.astype(np.float64)))
        got = rows_of(gdx, xd, rows, cols, ld)
        assert (np.abs(got - dx) <= bdx + HALF[xd] * (np.abs(dx) + bdx)).all(), k
        bw = (column_adds(rows, cols) + 2) * U * magw
        if accumulate:
            dw = dw + oldw.astype(np.float64)
            bw = bw + 2 * U * np.abs(dw)
        assert (np.abs(take(gdw, gd) - dw) <= bw + HALF[gd] * (np.abs(dw) + bw)).all(), k
        assert gdx.guards_intact() and gdw.guards_intact()


def test_backward_several_turns():
    """More rows than the strips take at once, in every form."""
    import torch
    z = zr()
    for rows, cols in ((40000, 96), (9001, 512), (9000, 1000), (2100, 2048), (2101, 4090), (1100, 8192), (700, 12001), (300, 16000)):
        g = torch.Generator("cuda").manual_seed(cols)
        h = torch.randn(rows, cols, generator=g, device="cuda").bfloat16()
        dy = torch.randn(rows, cols, generator=g, device="cuda").bfloat16()
        w = torch.randn(cols, generator=g, device="cuda")
        h64, d64 = h.double(), dy.double()
        rstd = (1 / torch.sqrt((h64 * h64).mean(1) + 1e-5)).float()
        dx, dw = torch.empty(rows, cols, device="cuda"), torch.empty(cols, device="cuda")
        ws = torch.empty(z.zr_rmsnorm_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
        z.zr_rmsnorm_bwd(dy, h, rows, cols, rstd, w, dx=dx, dweight=dw, workspace=ws)
        r = rstd.double()[:, None]
        xh, gg = h64 * r, d64 * w.double()
        c = (gg * xh).mean(1, keepdim=True)
        want = r * (gg - xh * c)
        lim = r * U * (2 * gg.abs() + 74 * xh.abs() * (gg * xh).abs().mean(1, keepdim=True)) + 3 * U * want.abs()
        assert bool(((dx.double() - want).abs() <= lim).all())
        want, mag = (d64 * xh).sum(0), (d64 * xh).abs().sum(0)
        assert bool(((dw.double() - want).abs() <= (column_adds(rows, cols) + 3) * U * mag).all())


def test_backward_is_the_forward_passes_slope():
    """Differences of the forward formula in 64 bits along random directions."""
    import torch
    z = zr()
    rng = np.random.default_rng(4)
    rows, cols, eps = 5, 700, 1e-5
    h, dy, w = (rng.standard_normal(s) for s in ((rows, cols), (rows, cols), cols))
    h, dy, w = (a.astype(np.float32).astype(np.float64) for a in (h, dy, w))
    f = lambda h, w: (h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * w * dy).sum()  # noqa: E731
    up = lambda a: torch.from_numpy(a.astype(np.float32)).cuda()  # noqa: E731
    y, rstd, dx, dw = torch.empty(rows, cols, device="cuda"), torch.empty(rows, device="cuda"), torch.empty(rows, cols, device="cuda"), \
        torch.empty(cols, device="cuda")
    z.zr_rmsnorm_fwd(up(h), rows, cols, y, up(w), eps=eps, rstd=rstd)
    ws = torch.empty(max(1, z.zr_rmsnorm_workspace_bytes(rows, cols)), dtype=torch.uint8, device="cuda")
    z.zr_rmsnorm_bwd(up(dy), up(h), rows, cols, rstd, up(w), dx=dx, dweight=dw, workspace=ws)
    for k in range(4):
        u, v = rng.standard_normal((rows, cols)), rng.standard_normal(cols)
        t = 1e-5
        slope = (f(h + t * u, w) - f(h - t * u, w)) / (2 * t)
        mine = (dx.cpu().numpy().astype(np.float64) * u).sum()
        assert abs(slope - mine) <= 1e-5 * np.abs(dx.cpu().numpy() * u).sum()
        slope = (f(h, w + t * v) - f(h, w - t * v)) / (2 * t)
        assert abs(slope - (dw.cpu().numpy().astype(np.float64) * v).sum()) <= 1e-5 * np.abs(dw.cpu().numpy() * v).sum()


def test_backward_in_place_parts_and_no_rows():
    import torch
    z = zr()
    for cols in (100, 4096, 13001):
        rows = 70
        h, dy = (torch.randn(rows, cols, device="cuda").bfloat16() for _ in range(2))
        w, rstd = torch.randn(cols, device="cuda"), torch.rand(rows, device="cuda") + 0.5
        ws = torch.empty(z.zr_rmsnorm_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
        dx, dw = torch.empty_like(h), torch.empty(cols, device="cuda")
        z.zr_rmsnorm_bwd(dy, h, rows, cols, rstd, w, dx=dx, dweight=dw, workspace=ws)
        only, onlyw = torch.empty_like(h), torch.empty(cols, device="cuda")
        z.zr_rmsnorm_bwd(dy, h, rows, cols, rstd, w, dx=only)
        z.zr_rmsnorm_bwd(dy, h, rows, cols, rstd, w, dweight=onlyw, workspace=ws)
        assert torch.equal(only, dx) and torch.equal(onlyw, dw)
        z.zr_rmsnorm_bwd(dy, h, rows, cols, rstd, w, dweight=onlyw, add_dx=True, workspace=ws)   # no dx to add to
        assert torch.equal(onlyw, dw)
        a, b = dy.clone(), h.clone()
        z.zr_rmsnorm_bwd(a, h, rows, cols, rstd, w, dx=a, dweight=onlyw, workspace=ws)
        z.zr_rmsnorm_bwd(dy, b, rows, cols, rstd, w, dx=b, dweight=onlyw, workspace=ws)
        assert torch.equal(a, dx) and torch.equal(b, dx) and torch.equal(onlyw, dw)
        empty = torch.empty(0, cols, dtype=torch.bfloat16, device="cuda")
        none = torch.empty(0, device="cuda")
        z.zr_rmsnorm_bwd(empty, empty, 0, cols, none, w, dx=empty, dweight=onlyw, accumulate=True, workspace=ws)
        assert torch.equal(onlyw, dw)
        z.zr_rmsnorm_bwd(empty, empty, 0, cols, none, w, dx=empty, dweight=onlyw, workspace=ws)
        assert bool((onlyw == 0).all())
        z.zr_rmsnorm_fwd(empty, 0, cols, empty, w, rstd=none)


def test_past_32_bits():
    """An element past 2^32, forward and backward: the last rows against the same rows alone."""
    import torch
    z = zr()
    cols = 4096
    rows = (1 << 32) // cols + 9
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-9:] = torch.randn(9, cols, device="cuda")
    y, rstd = torch.empty_like(x), torch.empty(rows, device="cuda")
    z.zr_rmsnorm_fwd(x, rows, cols, y, rstd=rstd)
    few, fr = torch.empty(9, cols, dtype=torch.bfloat16, device="cuda"), torch.empty(9, device="cuda")
    z.zr_rmsnorm_fwd(x[-9:], 9, cols, few, rstd=fr)
    assert torch.equal(y[-9:], few) and torch.equal(rstd[-9:], fr) and float(y[:-9].abs().max()) == 0
    z.zr_rmsnorm_bwd(y, x, rows, cols, rstd, dx=y)
    want = torch.empty_like(few)
    z.zr_rmsnorm_bwd(few, x[-9:], 9, cols, fr, dx=want)
    assert torch.equal(y[-9:], want)


def test_captured_and_on_a_stream():
    import torch
    z = zr()
    rows, cols = 900, 4096
    e = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    x, r, h, y, dy, dx = (e(rows, cols) for _ in range(6))
    w, rstd, dw = e(cols), e(rows, dt=torch.float32), e(cols, dt=torch.float32)
    cy = e(z.zr_ckpt_bytes(rows, cols), dt=torch.uint8)
    ws = e(z.zr_rmsnorm_workspace_bytes(rows, cols), dt=torch.uint8)

    def run():
        z.zr_rmsnorm_fwd(x, rows, cols, y, w, residual=r, h=h, rstd=rstd, ckpt_y=cy)
        z.zr_rmsnorm_bwd(dy, h, rows, cols, rstd, w, dx=dx, dweight=dw, workspace=ws)

    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    for t in (x, r, dy, w):
        t.copy_(torch.randn(t.shape, device="cuda"))
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        run()
    for seed in (1, 2, 3):
        g = torch.Generator("cuda").manual_seed(seed)
        for t in (x, r, dy, w):
            t.copy_(torch.randn(t.shape, device="cuda", generator=g))
        sides = []
        for how in range(3):
            for t in (h, y, dx, dw, rstd, cy):
                t.zero_()
            if how == 0:
                run()
            elif how == 1:
                graph.replay()
            else:
                stream.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(stream):
                    run()
                torch.cuda.current_stream().wait_stream(stream)
            torch.cuda.synchronize()
            sides.append([t.clone() for t in (h, y, dx, dw, rstd, cy)])
        assert all(torch.equal(a, b) for side in sides[1:] for a, b in zip(sides[0], side))
