"""Layer norm on the GPU against its formulas in 64 bits.

Bounds, with u = 2^-24 (half a step of fp32) and every sum of a row made of at
most 64 adds in line (a lane's own at most 32, then 6 across a wave and at most
8 across waves, or 16 across and 8 at a time in the wide form; the rest halves):
 * mean: 64 u mean|x|, and one division, so 66 u mean|x|;
 * the variance is a sum of squares of x - mean: 68 u of itself, so rstd is
   34 u off, its division and root 3 u more: 38 u rstd, plus the mean's error,
   which adds d^2 to the variance (d = 66 u mean|x|): below 38 u rstd wherever
   d <= 0.002 of the deviation, as in these inputs;
 * y: |w| rstd (66 u mean|x| + 2 u |x - mean|) + 40 u |w xh| + 2 u |y| + 2 u |w xh|,
   and half a step of y's type;
 * dx: written out below in the same way; dw, db: column_adds() u of the sum of
   magnitudes, and half a step of their type.
"""
import numpy as np
import pytest

import ckpt_ref as ref
from gpu_util import Guarded
from test_gpu_ckpt import bf16, tensor, to_bits16

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "fp32": U}


def zr():
    import gradient_sync_zr_amd as m
    return m


def code(dt):
    return {"bf16": zr().ZR_BF16, "fp32": zr().ZR_FP32, "e4m3": ref.E4M3, "int8": ref.INT8}[dt]


def td(dt):
    import torch
    return torch.bfloat16 if dt == "bf16" else torch.float32


def make(rng, rows, cols, dt, size=1.0):
    x = (rng.standard_normal((rows, cols)) * np.exp(0.5 * rng.standard_normal(cols)) + 0.3) * size
    x = x.astype(np.float32)
    return bf16(x) if dt == "bf16" else x


def vec(a, dt, shift=0):
    g = Guarded(a.size, td(dt), shift)
    g.set(to_bits16(a) if dt == "bf16" else a)
    return g


def take(g, dt):
    v = g.get()
    return (v.astype(np.uint32) << 16).view(np.float32) if dt == "bf16" else v


def rows_of(g, dt, rows, cols, ld, gap_value=None):
    v = np.concatenate([take(g, dt), np.full(ld - cols, 0.0 if gap_value is None else gap_value, np.float32)])
    v = v.reshape(rows, ld)
    if gap_value is not None:
        assert (v[:, cols:] == gap_value).all()
    return v[:, :cols].astype(np.float64)


def forward64(x, w, b, eps):
    mean = x.mean(1)
    var = ((x - mean[:, None]) ** 2).mean(1)
    rstd = 1 / np.sqrt(var + eps)
    xh = (x - mean[:, None]) * rstd[:, None]
    return xh * w + b, mean, rstd, xh


def forward_bounds(x, w, b, mean, rstd, xh, y, dt):
    m = 66 * U * np.abs(x).mean(1)
    r = 76 * U * rstd
    wxh = np.abs(w * xh)
    by = np.abs(w) * rstd[:, None] * (m[:, None] + 2 * U * np.abs(x - mean[:, None])) + 84 * U * wxh + 2 * U * np.abs(y)
    return m, r, by + HALF[dt] * (np.abs(y) + by)


# the register forms (16, 64, 256 and 512 lanes a row), their borders, and the wide form
COLS = [1, 2, 7, 8, 33, 100, 128, 129, 512, 515, 1000, 1024, 1025, 2048, 2100, 4096, 4104, 8192, 8200, 16384, 16385, 20011]


@pytest.mark.parametrize("cols", COLS)
def test_forward(cols):
    import torch
    z = zr()
    rng = np.random.default_rng(cols)
    for k, (rows, xd, yd, pd) in enumerate([(1, "bf16", "bf16", "bf16"), (37, "fp32", "bf16", "fp32"), (5, "bf16", "fp32", "fp32"),
                                            (18, "fp32", "fp32", "bf16"), (3, "e4m3", "bf16", "bf16"),
                                            (33, "int8", "fp32", "fp32")]):
        x = make(rng, rows, cols, "bf16" if xd != "fp32" else xd)
        w, b = make(rng, 1, cols, pd)[0], make(rng, 1, cols, pd)[0]
        affine = k != 3
        gap, shift = (5, 1) if k % 2 else (0, 0)
        x64 = x.astype(np.float64)
        if xd in ("e4m3", "int8"):
            src = torch.from_numpy(ref.buffer(*ref.pack(x64, code(xd)))).cuda()
            x64 = ref.held(x64, code(xd))
            held = None
        else:
            gx = tensor(x, xd, cols + gap, shift)
            src = gx.ptr()
            held = torch.full((ref.nbytes(rows, cols),), 0x55, dtype=torch.uint8, device="cuda")
        gw, gb = vec(w, pd, shift), vec(b, pd, shift)
        gy = Guarded((rows - 1) * (cols + gap) + cols, td(yd), shift)
        gy.t.fill_(3.0)
        gm, gr = Guarded(rows, torch.float32, shift), Guarded(rows, torch.float32)
        cy = torch.full((ref.nbytes(rows, cols),), 0x55, dtype=torch.uint8, device="cuda")
        fmt = (ref.E4M3, ref.INT8)[k % 2]
        eps = 1e-5 if cols > 2 else 0.1  # two columns: the variance may be anything
        z.zr_layernorm_fwd(src, rows, cols, gy.ptr(), gw.ptr() if affine else None, gb.ptr() if affine else None, eps=eps,
                           mean=gm.ptr(), rstd=gr.ptr(), ckpt_x=held, ckpt_y=cy, ckpt_format=fmt, x_dtype=code(xd),
                           y_dtype=code(yd), param_dtype=code(pd), ld_x=cols + gap, ld_y=cols + gap)
        w64, b64 = (w.astype(np.float64), b.astype(np.float64)) if affine else (np.ones(cols), np.zeros(cols))
        y, mean, rstd, xh = forward64(x64, w64, b64, eps)
        bm, br, by = forward_bounds(x64, w64, b64, mean, rstd, xh, y, yd)
        got = rows_of(gy, yd, rows, cols, cols + gap, 3.0)
        assert (np.abs(take(gm, "fp32") - mean) <= bm).all()
        assert (np.abs(take(gr, "fp32") - rstd) <= br).all()
        assert (np.abs(got - y) <= by).all()
        assert gy.guards_intact() and gm.guards_intact() and gr.guards_intact()
        # the checkpoints: of x exactly, and of y as it was written exactly
        if held is not None:
            assert np.array_equal(held.cpu().numpy(), ref.buffer(*ref.pack(x64, fmt)))
        assert np.array_equal(cy.cpu().numpy(), ref.buffer(*ref.pack(got, fmt)))


def test_forward_rows_of_one_value_and_not_finite():
    """A constant row has rstd = eps^-1/2 and y = bias; a row with a NaN or an infinity is NaN, others untouched by it."""
    import torch
    z = zr()
    for cols in (24, 300, 4096, 17000):
        x = np.ones((4, cols), np.float32) * 3
        x[1] = np.linspace(-1, 1, cols)
        x[2, cols // 2] = np.inf
        x[3, 0] = np.nan
        t = torch.from_numpy(x).cuda()
        y = torch.empty_like(t)
        mean, rstd = torch.empty(4, device="cuda"), torch.empty(4, device="cuda")
        b = torch.full((cols,), 0.5, device="cuda")
        z.zr_layernorm_fwd(t, 4, cols, y, bias=b, mean=mean, rstd=rstd, eps=1e-4)
        assert bool((y[0] == 0.5).all()) and float(mean[0]) == 3.0 and abs(float(rstd[0]) - 100) <= 100 * 4 * U
        assert bool(torch.isfinite(y[1]).all()) and bool(torch.isnan(y[2:]).all())


def test_forward_in_place_and_outputs_apart():
    import torch
    z = zr()
    for cols in (100, 4096, 17000):
        x = torch.randn(19, cols, device="cuda").bfloat16()
        want = torch.empty_like(x)
        z.zr_layernorm_fwd(x, 19, cols, want)
        m = torch.empty(19, device="cuda")
        z.zr_layernorm_fwd(x, 19, cols, mean=m)          # the statistics alone
        ck, cw = (torch.empty(z.zr_ckpt_bytes(19, cols), dtype=torch.uint8, device="cuda") for _ in range(2))
        z.zr_layernorm_fwd(x, 19, cols, ckpt_y=ck)       # the checkpoint alone: of y rounded to bf16
        z.zr_ckpt_pack(want, 19, cols, cw)
        assert torch.equal(ck, cw)
        wide = torch.full((19, 2 * cols), 9.0, device="cuda").bfloat16()
        wide[:, :cols] = x
        z.zr_layernorm_fwd(wide[:, :cols], 19, cols, wide[:, cols:])   # columns of one buffer
        assert torch.equal(wide[:, cols:], want) and torch.equal(wide[:, :cols], x)
        z.zr_layernorm_fwd(x, 19, cols, x)
        assert torch.equal(x, want)


# --------------------------------------------------------------- backward
def backward64(dy, x, mean, rstd, w):
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy * w
    n = x.shape[1]
    c1, c2 = (g * xh).sum(1) / n, g.sum(1) / n
    dx = rstd[:, None] * (g - c2[:, None] - xh * c1[:, None])
    mag = np.abs(g)
    bdx = rstd[:, None] * U * (5 * mag + 76 * mag.mean(1, keepdims=True) + 82 * np.abs(xh) * (mag * np.abs(xh)).mean(1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0), bdx, (np.abs(dy * xh)).sum(0), np.abs(dy).sum(0)


def column_adds(rows, cols):
    """Adds in line of a column's sum: a block takes `per` rows at once, each lane group the strip's share of
    them, then the groups' sums are added, then the strips' (16 groups of lanes, each every 16th, then those).
    At most 16384 elements are one block's, with more rows at once."""
    if rows * cols <= 16384:
        per = 64 if cols <= 128 else 16 if cols <= 512 else 8 if cols <= 1024 else 1
        return -(-rows // per) + min(per, rows)
    per = 16 if cols <= 128 else 4 if cols <= 1024 else 1
    steps = -(-rows // per)
    strips = min(steps, 512 if cols <= 4096 else 256)
    return -(-steps // strips) + per + -(-strips // 16) + 16


@pytest.mark.parametrize("cols", COLS)
def test_backward(cols):
    import torch
    z = zr()
    rng = np.random.default_rng(cols + 1)
    many = 1500 if cols <= 2100 else 520
    cases = [(1, "bf16", "bf16", "bf16", "bf16"), (37, "fp32", "fp32", "fp32", "fp32"), (many, "bf16", "bf16", "bf16", "fp32"),
             (18, "fp32", "bf16", "bf16", "bf16"), (3, "e4m3", "bf16", "fp32", "bf16"), (33, "int8", "fp32", "bf16", "fp32"),
             (many if cols < 9000 else 40, "e4m3", "fp32", "fp32", "fp32"), (21, "int8", "bf16", "bf16", "fp32")]
    for k, (rows, xd, dd, pd, gd) in enumerate(cases):
        x = make(rng, rows, cols, "bf16" if xd != "fp32" else xd)
        dy = make(rng, rows, cols, dd, 0.01)
        w = make(rng, 1, cols, pd)[0]
        affine, add, acc = k != 3, k % 3 == 1, k % 2 == 1
        gap, shift = (5, 1) if k % 2 else (0, 0)
        x64 = x.astype(np.float64)
        _, mean, rstd, _ = forward64(x64, 1.0, 0.0, 1e-5 if cols > 2 else 0.1)
        mean, rstd = mean.astype(np.float32), rstd.astype(np.float32)
        if xd in ("e4m3", "int8"):
            src = torch.from_numpy(ref.buffer(*ref.pack(x64, code(xd)))).cuda()
            x64 = ref.held(x64, code(xd))
        else:
            gx = tensor(x, xd, cols + gap, shift)
            src = gx.ptr()
        gdy = tensor(dy, dd, cols + gap, shift)
        gm, gr, gw = vec(mean, "fp32"), vec(rstd, "fp32", shift), vec(w, pd, shift)
        old = make(rng, rows, cols, dd, 0.01)
        gdx = tensor(old, dd, cols + gap, shift)
        ow, ob = make(rng, 1, cols, gd)[0], make(rng, 1, cols, gd)[0]
        gdw, gdb = vec(ow, gd, shift), vec(ob, gd, shift)
        nws = z.zr_layernorm_workspace_bytes(rows, cols)
        ws = torch.full((nws + 64,), 0xA5, dtype=torch.uint8, device="cuda")
        z.zr_layernorm_bwd(gdy.ptr(), src, rows, cols, gm.ptr(), gr.ptr(), gw.ptr() if affine else None, dx=gdx.ptr(),
                           dweight=gdw.ptr(), dbias=gdb.ptr(), accumulate=acc, add_dx=add, workspace=(ws.data_ptr(), nws),
                           dy_dtype=code(dd), x_dtype=code(xd), dx_dtype=code(dd), param_dtype=code(pd), grad_dtype=code(gd),
                           ld_dy=cols + gap, ld_x=cols + gap, ld_dx=cols + gap)
        dy64, w64 = dy.astype(np.float64), w.astype(np.float64) if affine else np.ones(cols)
        dx, dw, db, bdx, bw, bb = backward64(dy64, x64, mean.astype(np.float64), rstd.astype(np.float64), w64)
        if add:
            dx, bdx = dx + old, bdx + 2 * U * (np.abs(dx) + np.abs(old))
        got = rows_of(gdx, dd, rows, cols, cols + gap, 77.0)
        assert (np.abs(got - dx) <= bdx + HALF[dd] * (np.abs(dx) + bdx)).all(), k
        for g, want, mag, o in ((gdw, dw, bw, ow), (gdb, db, bb, ob)):
            want = want + (o if acc else 0)
            # three roundings of a term (x - mean, times rstd, times dy) and the column's adds
            lim = (column_adds(rows, cols) + 3) * U * mag + (2 * U * (mag + np.abs(o)) if acc else 0)
            assert (np.abs(take(g, gd) - want) <= lim + HALF[gd] * (np.abs(want) + lim)).all(), k
        for g in (gdx, gdw, gdb, gdy, gm, gr):
            assert g.guards_intact()
        assert bool((ws[nws:] == 0xA5).all())


def test_backward_against_differences():
    """dx, dw and db against central differences of the forward formula in 64 bits."""
    import torch
    z = zr()
    rng = np.random.default_rng(2)
    rows, cols, eps = 4, 40, 1e-3
    x, w, b, r = (rng.standard_normal(s).astype(np.float32) for s in ((rows, cols), cols, cols, (rows, cols)))
    t = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    y, mean, rstd = torch.empty(rows, cols, device="cuda"), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    z.zr_layernorm_fwd(t(x), rows, cols, y, t(w), t(b), eps=eps, mean=mean, rstd=rstd)
    dx, dw, db = torch.empty(rows, cols, device="cuda"), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    ws = torch.empty(z.zr_layernorm_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    z.zr_layernorm_bwd(t(r), t(x), rows, cols, mean, rstd, t(w), dx=dx, dweight=dw, dbias=db, workspace=ws)

    def loss(x_, w_, b_):
        return (forward64(x_, w_, b_, eps)[0] * r).sum()

    a = [v.astype(np.float64) for v in (x, w, b)]
    h = 1e-5  # the third derivative's term is about 1e-10, rounding 1e-11
    for got, which in ((dx, 0), (dw, 1), (db, 2)):
        got = got.cpu().numpy().astype(np.float64)
        for _ in range(12):
            at = tuple(rng.integers(0, n) for n in a[which].shape)
            up, dn = [v.copy() for v in a], [v.copy() for v in a]
            up[which][at] += h
            dn[which][at] -= h
            # fp32 results of sums of a few tens of terms of size 1
            assert abs((loss(*up) - loss(*dn)) / (2 * h) - got[at]) <= 1e-5 * (1 + abs(got[at]))


@pytest.mark.parametrize("cols", [100, 4096, 17000])
def test_backward_in_place_apart_and_without_rows(cols):
    import torch
    z = zr()
    rows = 41
    x, dy = torch.randn(rows, cols, device="cuda").bfloat16(), torch.randn(rows, cols, device="cuda").bfloat16()
    mean, rstd = x.float().mean(1), 1 / x.float().std(1)
    ws = torch.empty(z.zr_layernorm_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    new = lambda: torch.empty(cols, device="cuda")  # noqa: E731
    dx, dw, db = torch.empty_like(x), new(), new()
    z.zr_layernorm_bwd(dy, x, rows, cols, mean, rstd, dx=dx, dweight=dw, dbias=db, workspace=ws)
    only, w1, b1 = torch.empty_like(x), new(), new()
    z.zr_layernorm_bwd(dy, x, rows, cols, mean, rstd, dx=only)
    z.zr_layernorm_bwd(dy, x, rows, cols, mean, rstd, dweight=w1, workspace=ws)
    z.zr_layernorm_bwd(dy, x, rows, cols, mean, rstd, dbias=b1, workspace=ws)
    assert torch.equal(only, dx) and torch.equal(w1, dw) and torch.equal(b1, db)
    for place in ("dy", "x"):
        d2, x2, w2, b2 = dy.clone(), x.clone(), new(), new()
        z.zr_layernorm_bwd(d2, x2, rows, cols, mean, rstd, dx=d2 if place == "dy" else x2, dweight=w2, dbias=b2, workspace=ws)
        assert torch.equal(d2 if place == "dy" else x2, dx) and torch.equal(w2, dw) and torch.equal(b2, db)
    z.zr_layernorm_bwd(dy[:0], x[:0], 0, cols, mean[:0], rstd[:0], dx=only[:0], dweight=w2, accumulate=True, workspace=ws)
    assert torch.equal(w2, dw)
    z.zr_layernorm_bwd(dy[:0], x[:0], 0, cols, mean[:0], rstd[:0], dweight=w2, dbias=b2, workspace=ws)
    assert not w2.any() and not b2.any()


def test_offsets_past_32_bits():
    """More than 2^32 elements, in registers and in the wide form: the last rows equal a call of their own."""
    import torch
    z = zr()
    for rows, cols in ((530000, 8200), (66000, 65600)):
        x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
        for r in range(0, rows, rows // 10):
            x[r:r + rows // 10].normal_()
        y = torch.empty_like(x)
        ck = torch.empty(z.zr_ckpt_bytes(rows, cols), dtype=torch.uint8, device="cuda")
        mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        z.zr_layernorm_fwd(x, rows, cols, y, mean=mean, rstd=rstd, ckpt_x=ck)
        last, ly = x[-3:].clone(), torch.empty(3, cols, dtype=torch.bfloat16, device="cuda")
        lc = torch.empty(z.zr_ckpt_bytes(3, cols), dtype=torch.uint8, device="cuda")
        lm, lr = torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
        z.zr_layernorm_fwd(last, 3, cols, ly, mean=lm, rstd=lr, ckpt_x=lc)
        p = ref.pitch(cols)
        assert torch.equal(y[-3:], ly) and torch.equal(mean[-3:], lm) and torch.equal(rstd[-3:], lr)
        assert torch.equal(ck[(rows - 3) * p: rows * p], lc[:3 * p]) and torch.equal(ck[rows * p + (rows - 3) * (p // 32):], lc[3 * p:])
        z.zr_layernorm_bwd(y, ck, rows, cols, mean, rstd, dx=x, x_dtype=ref.E4M3)
        ldx = torch.empty_like(ly)
        z.zr_layernorm_bwd(ly, lc, 3, cols, lm, lr, dx=ldx, x_dtype=ref.E4M3)
        assert torch.equal(x[-3:], ldx)
        del x, y, ck
        torch.cuda.empty_cache()
