"""8-bit activation checkpoints on the GPU: pack and unpack bit for bit against
the 64-bit reference, and the weight gradient from a checkpoint.

Pack and unpack have one correct result for every input (one rounding of an
exact quotient; decoded values are exact in bf16), so they are compared bit for
bit. The weight gradient is compared exactly on inputs whose sums are exact in
fp32 in any order (small integers), and on others within the worst case of an
fp32 sum: products of bf16 values are exact in fp32 and each of the T + S adds
of T terms in S parts is off by at most one unit of 2^-23 of a partial sum that
no order makes larger than the sum of magnitudes (2^-24 if the matrix unit
rounds to nearest, 2^-23 should it truncate).
"""
import numpy as np
import pytest

import ckpt_ref as ref
from gpu_util import Guarded, bits, down16, up16

pytestmark = pytest.mark.gpu
FORMATS = [ref.E4M3, ref.INT8]


def zr():
    import gradient_sync_zr_amd as m
    return m


def bf16(x):
    """float32 array of bf16 values (truncated: any bf16 values will do)."""
    return (np.ascontiguousarray(x, dtype=np.float32).view(np.uint32) & 0xFFFF0000).view(np.float32)


def to_bits16(x):
    return (x.view(np.uint32) >> 16).astype(np.uint16)


def values(rng, rows, cols, dt):
    """Values over the whole range of fp32: blocks of very different sizes, borders of the formats, zeros of
    both signs, subnormals, a few blocks that are not finite."""
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-20, 20, (rows, cols)))
    e = rng.integers(-150, 128, (rows, -(-cols // 32))).repeat(32, 1)[:, :cols]
    x = np.where(rng.random((rows, 1)) < 0.5, x, rng.choice([-1.0, 1.0], x.shape) * (1 + rng.random(x.shape)) * np.exp2(e * 1.0))
    pick = rng.random((rows, cols))
    with np.errstate(over="ignore"):
        x = x.astype(np.float32)
    top = rng.choice([448.0, 127.0, 449.0, 126.5, 448.0 * 2 ** 119, 240.0 * 2.0 ** 120, 63.0 * 2.0 ** 122], (rows, cols))
    x = np.where(pick < 0.02, (top * np.exp2(rng.integers(-30, 1, x.shape) * 1.0)).astype(np.float32), x)
    x = np.where((pick > 0.02) & (pick < 0.05), np.float32(-0.0), x)
    x = np.where((pick > 0.05) & (pick < 0.07), np.float32(0.0), x)
    x = np.where(pick > 0.999, rng.choice([np.nan, np.inf, -np.inf], x.shape).astype(np.float32), x).astype(np.float32)
    return bf16(x) if dt == "bf16" else x


def tensor(x, dt, ld, shift=0):
    """A guarded device matrix with row stride ld holding x; returns (guard, address)."""
    import torch
    rows, cols = x.shape
    wide = np.full((rows, ld), 77.0, dtype=np.float32)
    wide[:, :cols] = x
    flat = wide.reshape(-1)[: (rows - 1) * ld + cols]
    g = Guarded(flat.size, torch.bfloat16 if dt == "bf16" else torch.float32, shift)
    g.set(to_bits16(flat) if dt == "bf16" else flat)
    return g


SHAPES = [(1, 1), (1, 32), (3, 33), (2, 7), (5, 64), (17, 1000), (64, 31), (9, 4096), (2, 20011), (1030, 40)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_pack_and_unpack_bit_for_bit(rows, cols, dt, fmt):
    import torch
    rng = np.random.default_rng(rows * 1000 + cols)
    code, td = (zr().ZR_BF16, torch.bfloat16) if dt == "bf16" else (zr().ZR_FP32, torch.float32)
    for gap, shift in ((0, 0), (3, 1)):
        x = values(rng, rows, cols, dt)
        g = tensor(x, dt, cols + gap, shift)
        n = ref.nbytes(rows, cols)
        guard = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        ck = guard[256: 256 + n]
        zr().zr_ckpt_pack(g.ptr(), rows, cols, ck, format=fmt, dtype=code, ld=cols + gap)
        codes, exps = ref.pack(x.astype(np.float64), fmt)
        got_c, got_e = ref.split(ck.cpu().numpy(), rows, cols)
        assert np.array_equal(got_e, exps)
        assert np.array_equal(got_c, codes)
        assert bool((guard[:256] == 0xA5).all()) and bool((guard[256 + n:] == 0xA5).all()) and g.guards_intact()
        # unpack into rows that are apart: the gaps keep what they hold
        out = Guarded((rows - 1) * (cols + gap) + cols, td, shift)
        out.t.fill_(3.0)
        zr().zr_ckpt_unpack(ck, rows, cols, out.ptr(), format=fmt, dtype=code, ld=cols + gap)
        want = ref.unpack(codes, exps, cols, fmt)
        got = out.get()
        got = (got.astype(np.uint32) << 16).view(np.float32) if dt == "bf16" else got
        got = np.concatenate([got, np.full(gap, 3.0, np.float32)]).reshape(rows, cols + gap)
        assert np.array_equal(got[:, :cols].astype(np.float64), want, equal_nan=True)
        finite = np.isfinite(want)
        assert np.array_equal(np.signbit(got[:, :cols])[finite], np.signbit(want)[finite]) or fmt == ref.INT8
        assert (got[:, cols:] == 3.0).all() and out.guards_intact()


@pytest.mark.parametrize("fmt", FORMATS)
def test_every_code_decodes(fmt):
    """All codes under all exponent bytes that packing writes, unpacked exactly to bf16."""
    import torch
    codes = np.tile(np.arange(256, dtype=np.uint8), (253, 1))
    if fmt == ref.E4M3:
        codes[:, [0x7F, 0xFF]] = 0
    exps = np.tile(np.arange(3, 256, dtype=np.uint8)[:, None], (1, 8))
    codes[252] = 0                                       # 255 comes with zero codes
    buf = torch.from_numpy(ref.buffer(codes, exps)).cuda()
    x = torch.empty(253, 256, dtype=torch.bfloat16, device="cuda")
    zr().zr_ckpt_unpack(buf, 253, 256, x, format=fmt)
    want = ref.unpack(codes, exps, 256, fmt)
    got = (down16(x).astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    ok = np.abs(want) < 2.0 ** 128                       # larger ones are not written by packing
    assert np.array_equal(got[ok], want[ok]) and np.isnan(got[252]).all()


def test_offsets_past_32_bits():
    """More than 2^32 elements: the last rows equal a pack of their own."""
    import torch
    rows, cols = 66000, 65536 + 32
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    for r in range(0, rows, 6000):
        x[r:r + 6000].normal_()
    ck = torch.empty(zr().zr_ckpt_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    zr().zr_ckpt_pack(x, rows, cols, ck, format=ref.INT8)
    one = torch.empty(zr().zr_ckpt_bytes(3, cols), dtype=torch.uint8, device="cuda")
    last = x[-3:].clone()
    zr().zr_ckpt_pack(last, 3, cols, one, format=ref.INT8)
    p = ref.pitch(cols)
    assert torch.equal(ck[(rows - 3) * p: rows * p], one[: 3 * p])
    assert torch.equal(ck[rows * p + (rows - 3) * (p // 32):], one[3 * p:])
    want = last.clone()
    zr().zr_ckpt_unpack(one, 3, cols, want, format=ref.INT8)
    zr().zr_ckpt_unpack(ck, rows, cols, x, format=ref.INT8)
    assert torch.equal(x[-3:], want)


# ------------------------------------------------------------ weight gradient
def run_wgrad(dy, x, fmt, dy_dt, grad_dt, bias, old=None, old_b=None, gaps=(0, 0), shift=0):
    """(dw, db) of the call on guarded buffers, as float32 arrays."""
    import torch
    rows, out, inn = dy.shape[0], dy.shape[1], x.shape[1]
    gd = tensor(dy, dy_dt, out + gaps[0], shift) if rows else None
    buf = torch.from_numpy(ref.buffer(*ref.pack(x.astype(np.float64), fmt))).cuda() if rows else 0
    ldw = inn + gaps[1]
    td = torch.bfloat16 if grad_dt == "bf16" else torch.float32
    gw = Guarded((out - 1) * ldw + inn, td, shift)
    gb = Guarded(out, td, shift)

    def put(g, a):
        g.set(to_bits16(a) if grad_dt == "bf16" else a)

    wide = np.full((out, ldw), 5.0, dtype=np.float32)
    wide[:, :inn] = 0.0 if old is None else old
    put(gw, wide.reshape(-1)[: gw.n])
    put(gb, np.zeros(out, np.float32) if old_b is None else old_b)
    z = zr()
    ws = torch.empty(z.zr_ckpt_wgrad_workspace_bytes(rows, out, inn) + 1, dtype=torch.uint8, device="cuda")
    z.zr_ckpt_wgrad(gd.ptr() if rows else 0, buf, rows, out, inn, gw.ptr(), dbias=gb.ptr() if bias else None, format=fmt,
                    accumulate=old is not None, workspace=ws, dy_dtype=z.ZR_BF16 if dy_dt == "bf16" else z.ZR_FP32,
                    grad_dtype=z.ZR_BF16 if grad_dt == "bf16" else z.ZR_FP32, ld_dy=out + gaps[0], ld_dw=ldw)

    def take(g):
        v = g.get()
        return (v.astype(np.uint32) << 16).view(np.float32) if grad_dt == "bf16" else v

    w = np.concatenate([take(gw), np.full(gaps[1], 5.0, np.float32)]).reshape(out, ldw)
    assert (w[:, inn:] == 5.0).all() and gw.guards_intact() and gb.guards_intact()
    if not bias:
        assert np.array_equal(take(gb), np.zeros(out, np.float32) if old_b is None else old_b)
    return w[:, :inn], take(gb)


WSHAPES = [(1, 1, 1), (1, 130, 40), (3, 16, 64), (63, 128, 128), (64, 129, 127), (65, 8, 300), (130, 257, 260), (513, 136, 72),
           (700, 300, 520), (1500, 40, 36)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dy_dt", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,out,inn", WSHAPES)
def test_wgrad_exact_on_integers(rows, out, inn, dy_dt, fmt):
    """|dy| <= 4 and |x| <= 8, integers: every partial sum is an integer below 2^24."""
    rng = np.random.default_rng(rows + 7 * out + 13 * inn)
    dy = rng.integers(-4, 5, (rows, out)).astype(np.float32)
    x = rng.integers(-8, 9, (rows, inn)).astype(np.float32)
    want = dy.astype(np.float64).T @ x.astype(np.float64)
    for gaps, shift, add in (((0, 0), 0, False), ((3, 5), 1, True), ((8, 0), 0, True)):
        old = rng.integers(-50, 50, (out, inn)).astype(np.float32) if add else None
        old_b = rng.integers(-50, 50, out).astype(np.float32) if add else None
        w, b = run_wgrad(dy, x, fmt, dy_dt, "fp32", True, old, old_b, gaps, shift)
        assert np.array_equal(w, want + (old if add else 0))
        assert np.array_equal(b, dy.sum(0) + (old_b if add else 0))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,out,inn", [(577, 136, 16384), (4160, 2056, 1090), (700, 4104, 4100), (65, 4104, 4100),
                                          (700, 4097, 4100), (65, 4103, 4100), (130, 4351, 4100),
                                          (9000, 2056, 1090), (4000, 4300, 4100)])
def test_wgrad_exact_on_integers_large(rows, out, inn, fmt):
    """The large form, with ragged last tiles and slabs, tiles split by rows (the last two sizes), and rows
    that do not start or end on 16 bytes."""
    rng = np.random.default_rng(rows)
    dy = rng.integers(-4, 5, (rows, out)).astype(np.float32)
    x = rng.integers(-8, 9, (rows, inn)).astype(np.float32)
    import torch
    want = (torch.from_numpy(dy).cuda().double().t() @ torch.from_numpy(x).cuda().double()).cpu().numpy()
    old = rng.integers(-50, 50, (out, inn)).astype(np.float32)
    for gaps, grad_dt, add in (((0, 0), "fp32", False), ((8, 3), "fp32", True), ((1, 0), "fp32", True), ((0, 5), "bf16", True)):
        w, b = run_wgrad(dy, x, fmt, "bf16", grad_dt, True, old if add else None, old[:, 0].copy() if add else None, gaps)
        exp_w, exp_b = want + (old if add else 0), dy.astype(np.float64).sum(0) + (old[:, 0] if add else 0)
        if grad_dt == "bf16":
            assert (np.abs(w - exp_w) <= 2.0 ** -8 * np.abs(exp_w)).all() and (np.abs(b - exp_b) <= 2.0 ** -8 * np.abs(exp_b)).all()
        else:
            assert np.array_equal(w, exp_w) and np.array_equal(b, exp_b)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dy_dt,grad_dt", [("bf16", "fp32"), ("bf16", "bf16"), ("fp32", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("rows,out,inn", [(37, 70, 100), (600, 264, 300), (1100, 130, 33)])
def test_wgrad_values(rows, out, inn, dy_dt, grad_dt, fmt):
    rng = np.random.default_rng(rows)
    dy = (rng.standard_normal((rows, out)) * np.exp(2 * rng.standard_normal((rows, 1)))).astype(np.float32)
    dy = bf16(dy) if dy_dt == "bf16" else dy
    x = bf16(rng.standard_normal((rows, inn)) * np.exp(rng.standard_normal(inn)))
    held = ref.held(x.astype(np.float64), fmt)
    old = bf16(rng.standard_normal((out, inn)))
    w, _ = run_wgrad(dy, x, fmt, dy_dt, grad_dt, False, old)
    want = dy.astype(np.float64).T @ held + old
    # adds: one per row (three per row for fp32 dy), one per part (at most 64), the old value; 2^-23 each
    n = rows * (3 if dy_dt == "fp32" else 1) + 66
    bound = n * 2.0 ** -23 * (np.abs(dy).astype(np.float64).T @ np.abs(held) + np.abs(old))
    if grad_dt == "bf16":
        bound += 2.0 ** -8 * np.abs(want)
    assert (np.abs(w - want) <= bound).all()
    # and as good as fp32 sums are in practice: their errors add up like a random walk
    rel = np.linalg.norm(w - want) / np.linalg.norm(want)
    assert rel <= (2.0 ** -8 if grad_dt == "bf16" else n ** 0.5 * 2.0 ** -23)


@pytest.mark.parametrize("fmt", FORMATS)
def test_wgrad_without_rows_and_values_that_are_not_finite(fmt):
    dy, x = np.zeros((0, 40), np.float32), np.zeros((0, 50), np.float32)
    w, b = run_wgrad(dy, x, fmt, "bf16", "fp32", True)
    assert not w.any() and not b.any()
    old = np.arange(2000, dtype=np.float32).reshape(40, 50)
    w, b = run_wgrad(dy, x, fmt, "bf16", "fp32", True, old, old[:, 0].copy())
    assert np.array_equal(w, old) and np.array_equal(b, old[:, 0])
    # a NaN block reaches its 32 columns only; an infinity in dy its own row of dw
    rng = np.random.default_rng(5)
    dy = rng.integers(-4, 5, (70, 40)).astype(np.float32)
    x = rng.integers(1, 9, (70, 100)).astype(np.float32)
    x[69, 40] = np.nan
    for dt in ("bf16", "fp32"):
        w, _ = run_wgrad(dy, x, fmt, dt, "fp32", False)
        assert np.isnan(w[:, 32:64]).all() and np.isfinite(w[:, :32]).all() and np.isfinite(w[:, 64:]).all()
        d2, x2 = dy.copy(), np.nan_to_num(x, nan=1.0)
        d2[69, 7] = np.inf
        w, b = run_wgrad(d2, x2, fmt, dt, "fp32", True)
        assert (w[7] == np.inf).all() and np.isfinite(np.delete(w, 7, 0)).all()
        assert b[7] == np.inf and np.isfinite(np.delete(b, 7)).all()


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_wgrad_offsets_past_32_bits(dt):
    """dy of more than 2^32 elements. Integers, and sums that wander far below 2^24, so exact in fp32."""
    import torch
    rows, out, inn = 1100000, 4096, 40
    dy = torch.empty(rows, out, dtype=torch.bfloat16 if dt == "bf16" else torch.float32, device="cuda")
    x = torch.randint(-8, 9, (rows, inn), device="cuda").float()
    want = torch.zeros(out, inn, dtype=torch.float64, device="cuda")
    step = 110000
    for r in range(0, rows, step):
        part = torch.randint(-4, 5, (step, out), device="cuda", dtype=torch.int8).float()
        dy[r:r + step] = part
        want += (part.t() @ x[r:r + step]).double()     # exact in fp32: at most 32 x 110,000
        del part
    ck = torch.empty(zr().zr_ckpt_bytes(rows, inn), dtype=torch.uint8, device="cuda")
    zr().zr_ckpt_pack(x, rows, inn, ck, format=ref.INT8)
    dw = torch.empty(out, inn, device="cuda")
    ws = torch.empty(zr().zr_ckpt_wgrad_workspace_bytes(rows, out, inn) + 1, dtype=torch.uint8, device="cuda")
    zr().zr_ckpt_wgrad(dy, ck, rows, out, inn, dw, format=ref.INT8, workspace=ws)
    assert torch.equal(dw.double(), want)
