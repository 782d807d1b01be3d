"""Layer norm on the GPU over more rows than a launch has places for, so that
every block goes over several (the next row's loads in flight, the slots of the
row sums used again), at the borders of every register form, and with dx of
another type than dy. Every row is compared with 64 bits, computed on the GPU.

test_gpu_norm_strided.py runs this module again with the grid capped at 13
blocks, where the kernels that have a block per row or tile stride too.

The bounds are those of test_gpu_norm.py (u = 2^-24); the forward's root is one
reciprocal root, off by one unit (2 u) where a root and a division would be off
by 3 u, and its means are products with 1 / n, 1 u more each.
"""
import os

import pytest

import ckpt_ref as ref
from gpu_util import Guarded

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
CAP = int(os.environ.get("ZR_MAX_GRID", 1 << 30))
HALF = {"bf16": 2.0 ** -8, "fp32": U}
# rows and columns: more than two turns of the 1024 blocks of 256 threads (512 of 512) for each register form,
# the last turn in part; then the wide form
FORMS = [(2 * 16384 + 37, 100), (2 * 4096 + 5, 500), (2 * 4096 + 7, 1000), (2 * 1024 + 3, 2041), (2 * 1024 + 3, 4088),
         (2 * 512 + 3, 8190), (2 * 512 + 3, 12288), (2 * 512 + 3, 16383), (53, 16390)]


def zr():
    import gradient_sync_zr_amd as m
    return m


def td(dt):
    import torch
    return torch.bfloat16 if dt == "bf16" else torch.float32


def gen(seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    import torch
    return torch.randn(*shape, generator=g, device="cuda")


def make(g, rows, cols, size=1.0):
    import torch
    return (randn(g, rows, cols) * torch.exp(0.5 * randn(g, cols)) + 0.3) * size


class Mat:
    """A guarded matrix whose rows are `gap` elements apart; the gaps hold 77."""

    def __init__(self, x, dt, gap=0, shift=0):
        import torch
        self.rows, self.cols = x.shape
        self.ld = self.cols + gap
        self.g = Guarded((self.rows - 1) * self.ld + self.cols, td(dt), shift)
        self.g.t.fill_(77.0)
        self.t = torch.as_strided(self.g.base, (self.rows, self.cols), (self.ld, 1), self.g.lo)
        self.t.copy_(x)

    def ok(self):
        import torch
        gaps = torch.ones(self.rows * self.ld, dtype=torch.bool, device="cuda").view(self.rows, self.ld)
        gaps[:, :self.cols] = False
        return self.g.guards_intact() and bool((self.g.t[gaps.view(-1)[:self.g.n]] == 77.0).all())


def ckpt(rows, cols):
    import torch
    return torch.full((zr().zr_ckpt_bytes(rows, cols),), 0x55, dtype=torch.uint8, device="cuda")


def held(ck, rows, cols, fmt):
    import torch
    x = torch.empty(rows, cols, device="cuda")
    zr().zr_ckpt_unpack(ck, rows, cols, x, format=fmt)
    return x


def packed(x, fmt):
    ck = ckpt(*x.shape)
    zr().zr_ckpt_pack(x, *x.shape, ck, format=fmt)
    return ck


def within(got, want, bound, what):
    import torch
    d = (got.double() - want).abs()
    bad = ~(d <= bound)
    assert not bool(bad.any()), (what, int(bad.sum()), torch.nonzero(bad)[:4].tolist())


@pytest.mark.parametrize("xd,yd,fmt", [("bf16", "bf16", ref.E4M3), ("fp32", "bf16", ref.INT8), ("bf16", "fp32", ref.INT8),
                                       ("e4m3", "bf16", ref.E4M3), ("int8", "fp32", ref.INT8)])
@pytest.mark.parametrize("rows,cols", FORMS)
def test_forward_over_many_rows(rows, cols, xd, yd, fmt):
    import torch
    z = zr()
    g = gen(rows + cols)
    x = make(g, rows, cols)
    gap, shift = (5, 1) if yd == "fp32" else (0, 0)
    w, b = (1 + 0.2 * randn(g, cols)).bfloat16(), randn(g, cols).bfloat16()
    cx = None
    if xd in ("e4m3", "int8"):
        f = ref.E4M3 if xd == "e4m3" else ref.INT8
        src = packed(x, f)
        x64, kx = held(src, rows, cols, f).double(), dict(x_dtype=f)
    else:
        m = Mat(x, xd, gap, shift)
        src, x64, kx, cx = m.t, m.t.double(), {}, ckpt(rows, cols)
    y = Mat(torch.zeros(rows, cols, device="cuda"), yd, gap, shift)
    mean, rstd = Guarded(rows, torch.float32, shift), Guarded(rows, torch.float32)
    cy = ckpt(rows, cols)
    z.zr_layernorm_fwd(src, rows, cols, y.t, w, b, eps=1e-5, mean=mean.ptr(), rstd=rstd.ptr(), ckpt_x=cx, ckpt_y=cy,
                       ckpt_format=fmt, **kx)
    torch.cuda.synchronize()
    m64 = x64.mean(1)
    c = x64 - m64[:, None]
    r64 = 1 / torch.sqrt((c * c).mean(1) + 1e-5)
    xh = c * r64[:, None]
    want = xh * w.double() + b.double()
    bm = 67 * U * x64.abs().mean(1)
    by = w.double().abs() * r64[:, None] * (bm[:, None] + 2 * U * c.abs()) + 84 * U * (w.double() * xh).abs() + \
        2 * U * want.abs()
    within(mean.t, m64, bm, "mean")
    within(rstd.t, r64, 76 * U * r64, "rstd")
    within(y.t, want, by + HALF[yd] * (want.abs() + by), "y")
    assert y.ok() and mean.guards_intact() and rstd.guards_intact()
    if cx is not None:
        assert torch.equal(cx, packed(src, fmt))
    assert torch.equal(cy, packed(y.t, fmt))
    if xd == yd:       # in place: the same bits
        keep = y.t.clone()
        z.zr_layernorm_fwd(src, rows, cols, src, w, b, eps=1e-5)
        torch.cuda.synchronize()
        assert torch.equal(src, keep)


def column_adds(rows, cols):
    """Adds in line of a column's sum, as in test_gpu_norm.py, under the grid's cap."""
    if rows * cols <= 16384:
        per = 64 if cols <= 128 else 16 if cols <= 512 else 8 if cols <= 1024 else 1
        return -(-rows // per) + min(per, rows)
    per = 16 if cols <= 128 else 4 if cols <= 1024 else 1
    steps = -(-rows // per)
    strips = min(steps, 512 if cols <= 4096 else 256, CAP)
    return -(-steps // strips) + per + -(-strips // 16) + 16


BWD = [(3, 100), (2 * 8192 + 37, 100), (4133, 500), (4135, 1000), (1027, 2041), (1027, 4088), (519, 8190), (519, 12281),
       (519, 12288), (519, 12289), (300, 16383)]


@pytest.mark.parametrize("xd,dd,od,gd", [("bf16", "bf16", "fp32", "bf16"), ("fp32", "fp32", "bf16", "fp32"),
                                         ("e4m3", "bf16", "fp32", "fp32"), ("int8", "fp32", "bf16", "bf16"),
                                         ("fp32", "bf16", "fp32", "fp32"), ("bf16", "fp32", "bf16", "fp32"),
                                         ("bf16", "bf16", "bf16", "bf16")])
@pytest.mark.parametrize("rows,cols", BWD)
def test_backward_over_many_rows(rows, cols, xd, dd, od, gd):
    """od: dx's type. Each pair of types with dx and the gradients overwritten and added to."""
    import torch
    z = zr()
    g = gen(rows + cols)
    x = make(g, rows, cols)
    x = x.bfloat16().float() if xd != "fp32" else x
    m64 = x.double().mean(1)
    rstd = (1 / torch.sqrt(((x.double() - m64[:, None]) ** 2).mean(1) + 1e-5)).float()
    mean = m64.float()
    w = 1 + 0.2 * randn(g, cols)
    if xd in ("e4m3", "int8"):
        f = ref.E4M3 if xd == "e4m3" else ref.INT8
        src = packed(x, f)
        x64, kx = held(src, rows, cols, f).double(), dict(x_dtype=f)
    else:
        src = Mat(x, xd, 3, 1).t
        x64, kx = src.double(), {}
    n = z.zr_layernorm_workspace_bytes(rows, cols)
    for add in (False, True):
        gap, shift = (5, 1) if add else (0, 0)
        dy = Mat(make(g, rows, cols, 0.01), dd, gap, shift)
        old = make(g, rows, cols, 0.01).to(td(od))
        dx = Mat(old, od, gap, shift)
        ow, ob = randn(g, cols).to(td(gd)), randn(g, cols).to(td(gd))
        gw, gb = Guarded(cols, td(gd), shift), Guarded(cols, td(gd), shift)
        gw.t.copy_(ow)
        gb.t.copy_(ob)
        ws = torch.full((n + 64,), 0xA5, dtype=torch.uint8, device="cuda")
        z.zr_layernorm_bwd(dy.t, src, rows, cols, mean, rstd, w, dx=dx.t, dweight=gw.ptr(), dbias=gb.ptr(), accumulate=add,
                           add_dx=add, workspace=(ws.data_ptr(), n), grad_dtype=td(gd), **kx)
        torch.cuda.synchronize()
        r64 = rstd.double()[:, None]
        xh = (x64 - mean.double()[:, None]) * r64
        d64 = dy.t.double()
        gy = d64 * w.double()
        want = r64 * (gy - gy.mean(1, keepdim=True) - xh * (gy * xh).mean(1, keepdim=True))
        mag = gy.abs()
        bound = r64 * U * (5 * mag + 76 * mag.mean(1, keepdim=True) + 82 * xh.abs() * (mag * xh.abs()).mean(1, keepdim=True))
        if add:
            want = want + old.double()
            bound = bound + 2 * U * (want.abs() + old.double().abs())
        within(dx.t, want, bound + HALF[od] * (want.abs() + bound), ("dx", add))
        for got, terms, o, what in ((gw.t, d64 * xh, ow, "dweight"), (gb.t, d64, ob, "dbias")):
            want, mag = terms.sum(0), terms.abs().sum(0)
            bound = (column_adds(rows, cols) + 3) * U * mag
            if add:
                want, bound = want + o.double(), bound + 2 * U * (mag + o.double().abs())
            within(got, want, bound + HALF[gd] * (want.abs() + bound), (what, add))
        assert dx.ok() and dy.ok() and gw.guards_intact() and gb.guards_intact() and bool((ws[n:] == 0xA5).all())


def test_rows_and_columns_past_the_launch_limit():
    """Sizes at which a block per row or per 64 columns would be 2^32 threads or more: the last rows, and every
    column, equal calls of their own."""
    import torch
    z = zr()
    cols = 1 << 27
    x, dy = torch.empty(2, cols, device="cuda").bfloat16(), torch.empty(2, cols, device="cuda").bfloat16()
    x.normal_(generator=gen(1))
    dy.normal_(generator=gen(2))
    dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    mean, rstd = torch.tensor([0.5, -0.25], device="cuda"), torch.tensor([2.0, 0.5], device="cuda")
    ws = torch.empty(z.zr_layernorm_workspace_bytes(2, cols), dtype=torch.uint8, device="cuda")
    z.zr_layernorm_bwd(dy, x, 2, cols, mean, rstd, dweight=dw, dbias=db, workspace=ws)
    # two terms, each of them and their sum rounded once
    assert torch.equal(db, dy[0].float() + dy[1].float())
    for lo in range(0, cols, cols // 8):
        s = slice(lo, lo + cols // 8)
        xh = (x[:, s].double() - mean.double()[:, None]) * rstd.double()[:, None]
        terms = xh * dy[:, s].double()
        within(dw[s], terms.sum(0), 5 * U * terms.abs().sum(0), "dweight")
    del x, dy, dw, db, ws
    torch.cuda.empty_cache()
    rows, cols = (1 << 22) + 5, 12300       # (the forward's wide form starts at 16385)
    p = ref.pitch(cols)
    ck = torch.zeros(z.zr_ckpt_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    ck[rows * p:] = 127
    last = packed(randn(gen(3), 7, cols), ref.INT8)
    ck[(rows - 7) * p: rows * p] = last[:7 * p]
    ck[rows * p + (rows - 7) * (p // 32):] = last[7 * p:]
    dx = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    dx[-7:] = randn(gen(4), 7, cols)
    mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    want = dx[-7:].clone()
    z.zr_layernorm_bwd(want, last, 7, cols, mean[:7], rstd[:7], dx=want, x_dtype=ref.INT8)
    z.zr_layernorm_bwd(dx, ck, rows, cols, mean, rstd, dx=dx, x_dtype=ref.INT8)
    assert torch.equal(dx[-7:], want) and not bool(dx[:1000].any()) and not bool(dx[rows // 2: rows // 2 + 1000].any())
    del dx, ck
    torch.cuda.empty_cache()
    cols = 16400
    p = ref.pitch(cols)
    ck = torch.zeros(z.zr_ckpt_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    ck[rows * p:] = 127
    last = packed(randn(gen(5), 7, cols) + 0.5, ref.INT8)
    ck[(rows - 7) * p: rows * p] = last[:7 * p]
    ck[rows * p + (rows - 7) * (p // 32):] = last[7 * p:]
    mean.fill_(9.0)
    rstd.fill_(9.0)
    z.zr_layernorm_fwd(ck, rows, cols, mean=mean, rstd=rstd, x_dtype=ref.INT8, eps=0.25)
    m, r = torch.empty(7, device="cuda"), torch.empty(7, device="cuda")
    z.zr_layernorm_fwd(last, 7, cols, mean=m, rstd=r, x_dtype=ref.INT8, eps=0.25)
    assert torch.equal(mean[-7:], m) and torch.equal(rstd[-7:], r)
    assert not bool(mean[:-7].any()) and bool((rstd[:-7] == 2.0).all())
    del ck
    torch.cuda.empty_cache()
