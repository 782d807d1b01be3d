"""4-bit blocks, and transposes packed in every format, on the GPU: bit for bit with
the 64-bit reference."""
import numpy as np
import pytest

import pack_ref as pk
from gpu_util import Guarded, bits
from test_gpu_grads import bf16

pytestmark = pytest.mark.gpu


def zr():
    import gradient_sync_zr_amd as m
    return m


def upload(x, dt, ld, shift=0):
    """rows of x at a stride of ld elements, NaN between them."""
    import torch
    rows, cols = x.shape
    g = Guarded((rows - 1) * ld + cols, torch.bfloat16 if dt == "bf16" else torch.float32, shift)
    g.t.fill_(float("nan"))
    g.t.as_strided((rows, cols), (ld, 1)).copy_(torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda())
    return g


def buffer(rows, cols, fmt, value=0x55):
    import torch
    return torch.full((pk.nbytes(rows, cols, fmt) + 64,), value, dtype=torch.uint8, device="cuda")


def make(rng, rows, cols, dt):
    x = (rng.standard_normal((rows, cols)) * np.exp(3 * rng.standard_normal((rows, 1)))).astype(np.float32)
    x[rng.random(x.shape) < 0.05] = 0.0
    return bf16(x) if dt == "bf16" else x


SIZES = [(1, 1), (1, 31), (3, 32), (5, 33), (33, 95), (7, 1000), (129, 64), (64, 257), (31, 4096), (1000, 300)]


@pytest.mark.parametrize("rows,cols", SIZES)
def test_pack_and_unpack(rows, cols):
    import torch
    z = zr()
    rng = np.random.default_rng(rows * 7 + cols)
    for dt, gap, shift in (("bf16", 0, 0), ("fp32", 0, 0), ("bf16", 5, 1), ("fp32", 3, 1)):
        code = z.ZR_BF16 if dt == "bf16" else z.ZR_FP32
        x = make(rng, rows, cols, dt)
        g = upload(x, dt, cols + gap, shift)
        out = buffer(rows, cols, pk.E2M1)
        z.zr_ckpt_pack(g.ptr(), rows, cols, out, format=pk.E2M1, dtype=code, ld=cols + gap)
        want = pk.pack(x.astype(np.float64), pk.E2M1)
        got = out.cpu().numpy()
        assert np.array_equal(got[:want.size], want) and (got[want.size:] == 0x55).all()
        for back, bcode in ((torch.bfloat16, z.ZR_BF16), (torch.float32, z.ZR_FP32)):
            y = Guarded((rows - 1) * (cols + gap) + cols, back, shift)
            y.t.fill_(7.0)
            z.zr_ckpt_unpack(out, rows, cols, y.ptr(), format=pk.E2M1, dtype=bcode, ld=cols + gap)
            v = torch.cat([y.t, torch.full((gap,), 7.0, dtype=back, device="cuda")]).view(rows, cols + gap).float().cpu().numpy()
            held = pk.unpack(want, rows, cols, pk.E2M1).astype(np.float32)
            assert np.array_equal(bits(np.ascontiguousarray(v[:, :cols])), bits(np.ascontiguousarray(held)))
            assert (v[:, cols:] == 7.0).all() and y.guards_intact()


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_every_bf16_value(dt):
    """Each of the 2^16 patterns beside a larger one by 2^0 to 2^9 and a half more, in rows without gaps and with."""
    import torch
    z = zr()
    v = (np.arange(1 << 16, dtype=np.uint32) << 16).view(np.float32)
    with np.errstate(all="ignore"):
        most = (np.abs(v)[:, None] * 2.0 ** np.arange(10, dtype=np.float32) * np.float32(1.5)).astype(np.float32)
    most[most > 3.0e38] = 3.0e38
    x = np.zeros((1 << 16, 10, 32), np.float32)
    x[:, :, 7], x[:, :, 30] = v[:, None], bf16(most)
    x = x.reshape(1 << 15, 640)
    code = z.ZR_BF16 if dt == "bf16" else z.ZR_FP32
    want = pk.pack(x.astype(np.float64), pk.E2M1)
    for gap, shift in ((0, 0), (0, 3), (5, 0)):
        g = upload(x, dt, 640 + gap, shift)
        out = buffer(1 << 15, 640, pk.E2M1)
        z.zr_ckpt_pack(g.ptr(), 1 << 15, 640, out, format=pk.E2M1, dtype=code, ld=640 + gap)
        got = out.cpu().numpy()
        assert np.array_equal(got[:want.size], want) and (got[want.size:] == 0x55).all()
    y = torch.empty(1 << 15, 640, dtype=torch.bfloat16 if dt == "bf16" else torch.float32, device="cuda")
    z.zr_ckpt_unpack(out, 1 << 15, 640, y, format=pk.E2M1)
    held = pk.unpack(want, 1 << 15, 640, pk.E2M1).astype(np.float32)
    got, nan = y.float().cpu().numpy(), np.isnan(held)
    assert np.array_equal(np.isnan(got), nan) and np.array_equal(bits(got)[~nan], bits(held)[~nan])


@pytest.mark.parametrize("rows,cols", SIZES + [(4096, 70), (300, 1100)])
def test_transposed(rows, cols):
    z = zr()
    rng = np.random.default_rng(rows * 11 + cols)
    for k, fmt in enumerate((pk.E4M3, pk.INT8, pk.E2M1)):
        for dt, gap, shift in (("bf16", 0, 0), ("fp32", 6, 1)):
            x = make(rng, rows, cols, dt)
            g = upload(x, dt, cols + gap, shift)
            out = buffer(cols, rows, fmt)
            z.zr_ckpt_pack_t(g.ptr(), rows, cols, out, format=fmt, dtype=z.ZR_BF16 if dt == "bf16" else z.ZR_FP32,
                             ld=cols + gap)
            want = pk.pack(np.ascontiguousarray(x.T).astype(np.float64), fmt)
            got = out.cpu().numpy()
            assert np.array_equal(got[:want.size], want) and (got[want.size:] == 0x55).all()


@pytest.mark.parametrize("rows,cols", [(2070, 16200), (4100, 8200), (2 * 32 * 2049, 250)])
def test_transposed_large(rows, cols):
    """Enough tiles that a lane takes several blocks, the last lanes fewer: as the transpose packed by rows."""
    import torch
    z = zr()
    g = torch.Generator("cuda").manual_seed(rows)
    for dt in (torch.bfloat16, torch.float32):
        x = (torch.randn(rows, cols + 3, generator=g, device="cuda") * torch.exp(2 * torch.randn(rows, 1, generator=g, device="cuda"))).to(dt)
        x[5, 7], x[rows - 1, cols - 1] = float("nan"), float("inf")
        x, xt = x[:, :cols], x[:, :cols].t().contiguous()
        for fmt in (pk.E2M1, pk.E4M3, z.ZR_CKPT_INT8):
            n = z.zr_ckpt_format_bytes(cols, rows, fmt)
            got, want = (torch.full((n + 64,), 0x55, dtype=torch.uint8, device="cuda") for _ in range(2))
            z.zr_ckpt_pack_t(x, rows, cols, got, format=fmt, ld=cols + 3)
            z.zr_ckpt_pack(xt, cols, rows, want, format=fmt)
            assert torch.equal(got, want)


def test_special_values():
    """Zeros of both signs, subnormals, the largest values, NaN and infinities, ties, each in a block of its own."""
    import torch
    z = zr()
    f = np.float32
    top, tiny = np.finfo(f).max, f(2.0 ** -149)
    blocks = [[0.0], [-0.0, 0.0], [tiny, -tiny], [2.0 ** -126, 2.0 ** -127], [top, 1.0, -top], [2.0 ** 127, -1.75 * 2.0 ** 127],
              [np.nan, 1.0], [np.inf, 2.0], [-np.inf], [6.0, 5.0, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -5.0, -0.25],
              [6.000001, 1.0], [2.0 ** 126, 3.5 * 2.0 ** 125]]
    x = np.zeros((len(blocks), 32), f)
    for k, b in enumerate(blocks):
        x[k, :len(b)] = b
    x[1, 2:] = -0.0
    t = torch.from_numpy(x).cuda()
    want = pk.pack(x.astype(np.float64), pk.E2M1)
    out = torch.zeros(want.size, dtype=torch.uint8, device="cuda")
    z.zr_ckpt_pack(t, *x.shape, out, format=pk.E2M1)
    assert np.array_equal(out.cpu().numpy(), want)
    z.zr_ckpt_pack_t(t.t().contiguous(), 32, len(blocks), out, format=pk.E2M1)
    assert np.array_equal(out.cpu().numpy(), want)
    y = torch.empty_like(t)
    z.zr_ckpt_unpack(out, *x.shape, y, format=pk.E2M1)
    assert np.array_equal(y.cpu().numpy(), pk.unpack(want, *x.shape, pk.E2M1).astype(f), equal_nan=True)
    b = t.bfloat16()
    z.zr_ckpt_pack(b, *x.shape, out, format=pk.E2M1)
    assert np.array_equal(out.cpu().numpy(), pk.pack(b.float().cpu().numpy().astype(np.float64), pk.E2M1))


def test_past_32_bits():
    """Codes and elements past 2^32."""
    import torch
    z = zr()
    rows, cols = (1 << 32) // 4096 + 17, 4096
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-1] = torch.arange(cols, device="cuda").bfloat16()
    x[-2, 5] = 3.0
    out = torch.empty(pk.nbytes(rows, cols, pk.E2M1), dtype=torch.uint8, device="cuda")
    z.zr_ckpt_pack(x, rows, cols, out, format=pk.E2M1)
    want = pk.held(x[-3:].float().cpu().numpy().astype(np.float64), pk.E2M1)
    x.fill_(1.0)
    z.zr_ckpt_unpack(out, rows, cols, x, format=pk.E2M1)
    assert np.array_equal(x[-3:].float().cpu().numpy(), want) and int((x[:-2] != 0).sum()) == 0
    # the transpose of 64 columns: rows past 2^26 each
    tall = x.view(-1, 64)
    n = tall.shape[0]
    big = torch.empty(pk.nbytes(64, n, pk.E4M3), dtype=torch.uint8, device="cuda")
    z.zr_ckpt_pack_t(tall, n, 64, big)
    p = -(-n // 32) * 32
    codes, exps = big[:64 * p].view(64, p), big[64 * p:].view(64, p // 32)
    last = tall[-32:].float().cpu().numpy().astype(np.float64).T
    ref = pk.pack(np.ascontiguousarray(last), pk.E4M3)
    assert n % 32 == 0 and np.array_equal(codes[:, -32:].cpu().numpy(), ref[:64 * 32].reshape(64, 32))
    assert np.array_equal(exps[:, -1].cpu().numpy(), ref[64 * 32:])
