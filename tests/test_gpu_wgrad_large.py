"""The weight gradient's large form (tiles of 256 x 256) on the GPU: every size
here takes it (test_wgrad_forms_cpu.py asserts that), whole and with tiles split
by rows, with last tiles, chunks and slabs in part; and both forms' decoding at
every exponent.

Exact comparisons use integers whose partial sums stay below 2^24; others the
worst case of an fp32 sum, as in test_gpu_ckpt.py: one unit of 2^-23 of the sum
of magnitudes for each add (one per row, one per part, one for an old value).
References are products in 64 bits on the GPU.
"""
import numpy as np
import pytest

import ckpt_ref as ref
from gpu_util import Guarded

pytestmark = pytest.mark.gpu
FORMATS = [ref.E4M3, ref.INT8]

# rows, out, in: whole tiles only (False) or with some tiles split by rows (True)
WHOLE = [(65, 4104, 4100), (700, 4097, 4100), (130, 4351, 4100)]
SPLIT = [(4000, 4300, 4100), (200000, 40, 70), (300000, 8, 33), (300001, 131, 257)]
FAR = (1100000, 4096, 512)       # dY of more than 2^32 elements
EXPONENTS = (253, 4351, 4100)    # rows under all exponent bytes
SMALL_EXPONENTS = (253, 260, 300)


def zr():
    import gradient_sync_zr_amd as m
    return m


def rand_int(g, shape, most):
    import torch
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda", dtype=torch.int8)


def gen(seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def pack(x, fmt):
    import torch
    z = zr()
    ck = torch.empty(z.zr_ckpt_bytes(*x.shape), dtype=torch.uint8, device="cuda")
    z.zr_ckpt_pack(x.contiguous(), *x.shape, ck, format=fmt)
    return ck


def held(ck, rows, cols, fmt):
    import torch
    x = torch.empty(rows, cols, device="cuda")
    zr().zr_ckpt_unpack(ck, rows, cols, x, format=fmt)
    return x


def product64(dy, x):
    """dy^T x in 64 bits, over slices of the rows."""
    import torch
    want = torch.zeros(dy.shape[1], x.shape[1], dtype=torch.float64, device="cuda")
    for r in range(0, dy.shape[0], 1 << 16):
        want += dy[r:r + (1 << 16)].double().t().contiguous() @ x[r:r + (1 << 16)].double()
    return want


def wgrad(dy, ck, inn, fmt, grad=None, old=None, old_b=None, gap=0, shift=0):
    """dw, db (float32) of the call with guarded gradients, rows of dw `gap` apart."""
    import torch
    z = zr()
    rows, out = dy.shape
    td = grad or torch.float32
    ldw = inn + gap
    gw, gb = Guarded((out - 1) * ldw + inn, td, shift), Guarded(out, td, shift)
    wide = torch.full((out, ldw), 5.0, device="cuda")
    wide[:, :inn] = 0 if old is None else old
    gw.t.copy_(wide.reshape(-1)[:gw.n])
    gb.t.copy_(torch.zeros(out, device="cuda") if old_b is None else old_b)
    n = z.zr_ckpt_wgrad_workspace_bytes(rows, out, inn)
    ws = torch.full((n + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    z.zr_ckpt_wgrad(dy, ck, rows, out, inn, gw.ptr(), dbias=gb.ptr(), format=fmt, accumulate=old is not None,
                    workspace=(ws.data_ptr(), n), grad_dtype=td, ld_dw=ldw)
    torch.cuda.synchronize()
    assert gw.guards_intact() and gb.guards_intact() and bool((ws[n:] == 0xA5).all())
    w = torch.full((out * ldw,), 5.0, device="cuda")
    w[:gw.n] = gw.t.float()
    w = w.view(out, ldw)
    assert bool((w[:, inn:] == 5.0).all())
    return w[:, :inn], gb.t.float()


def say(*a):
    print(*a, flush=True)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,out,inn", WHOLE + SPLIT)
def test_exact_on_integers(rows, out, inn, fmt):
    """|dy| <= 1 and |x| <= 8: a sum of 300,000 products stays below 2^24, and old values are small. Strided dy,
    and dw and db at odd addresses."""
    import torch
    g = gen(rows + out)
    x = rand_int(g, (rows, inn), 8).float()
    ck = pack(x, fmt)
    for gap, shift, add, pad in ((0, 0, False, 0), (3, 1, True, 5), (0, 0, True, 8)):
        wide = rand_int(g, (rows, out + pad), 1).bfloat16()
        dy = wide[:, :out]
        want, want_b = product64(dy, x), dy.double().sum(0)
        old = rand_int(g, (out, inn), 50).float() if add else None
        old_b = rand_int(g, (out,), 50).float() if add else None
        w, b = wgrad(dy, ck, inn, fmt, None, old, old_b, gap, shift)
        assert torch.equal(w.double(), want + (old if add else 0))
        assert torch.equal(b.double(), want_b + (old_b if add else 0))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("grad", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,out,inn", [(700, 4097, 4100), (4000, 4300, 4100), (300001, 131, 257)])
def test_values(rows, out, inn, grad, fmt):
    import torch
    g = gen(rows)
    td = torch.bfloat16 if grad == "bf16" else torch.float32
    dy = (torch.randn(rows, out, generator=g, device="cuda") *
          torch.exp(torch.randn(rows, 1, generator=g, device="cuda"))).bfloat16()
    x = (torch.randn(rows, inn, generator=g, device="cuda") *
         torch.exp(torch.randn(inn, generator=g, device="cuda"))).bfloat16()
    old = torch.randn(out, inn, generator=g, device="cuda").to(td).float()
    old_b = torch.randn(out, generator=g, device="cuda").to(td).float()
    ck = pack(x, fmt)
    hx = held(ck, rows, inn, fmt)
    w, b = wgrad(dy, ck, inn, fmt, td, old, old_b)
    n = rows + 258     # parts are at most 256
    for got, want, mag in ((w, product64(dy, hx) + old, product64(dy.abs(), hx.abs()) + old.abs()),
                           (b, dy.double().sum(0) + old_b, dy.double().abs().sum(0) + old_b.abs())):
        bound = n * 2.0 ** -23 * mag
        if grad == "bf16":
            bound = bound + 2.0 ** -8 * (want.abs() + bound)
        assert bool(((got - want).abs() <= bound).all())
        rel = float(torch.linalg.norm(got - want) / torch.linalg.norm(want))
        say(rows, out, inn, grad, fmt, "relative", rel)
        assert rel <= (2.0 ** -8 if grad == "bf16" else n ** 0.5 * 2.0 ** -23)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,out,inn", [(700, 4097, 4100), (65, 4104, 4100), (4000, 4300, 4100), (300001, 131, 257)])
def test_values_that_are_not_finite(rows, out, inn, fmt):
    """A block that is not finite reaches its own columns only, wherever it lies (the last row, the last block in
    part, a first tile's edge); an infinity or a NaN of dy its own row of dw and its own db."""
    import torch
    g = gen(3)
    x = torch.randint(1, 9, (rows, inn), generator=g, device="cuda").float()
    dy = torch.randint(1, 5, (rows, out), generator=g, device="cuda").bfloat16()
    last = (inn - 1) // 32 * 32
    for r, c, bad in ((rows - 1, inn - 1, float("nan")), (0, 0, float("inf")), (rows // 2, min(255, inn - 1), -float("inf")),
                      (63, last, float("nan"))):
        x2 = x.clone()
        x2[r, c] = bad
        w, b = wgrad(dy, pack(x2, fmt), inn, fmt)
        block = torch.zeros(inn, dtype=torch.bool, device="cuda")
        block[c // 32 * 32: c // 32 * 32 + 32] = True
        assert bool(torch.isnan(w[:, block]).all()) and bool(torch.isfinite(w[:, ~block]).all())
        assert bool(torch.isfinite(b).all())
    ck = pack(x, fmt)
    for r, c, bad in ((rows - 1, out - 1, float("inf")), (0, 0, -float("inf")), (rows - 1, out - 2, float("nan")),
                      (min(64, rows - 1), min(out - 1, 128), float("inf"))):
        d2 = dy.clone()
        d2[r, c] = bad
        w, b = wgrad(d2, ck, inn, fmt)
        own = torch.zeros(out, dtype=torch.bool, device="cuda")
        own[c] = True
        want = torch.full((), bad, device="cuda")
        assert torch.allclose(w[own], want, equal_nan=True) and torch.allclose(b[own], want, equal_nan=True)
        assert bool(torch.isfinite(w[~own]).all()) and bool(torch.isfinite(b[~own]).all())


def test_offsets_past_32_bits():
    """dy of more than 2^32 elements; |dy| <= 1 and |x| <= 8, so sums stay below 2^24."""
    import torch
    rows, out, inn = FAR
    g = gen(9)
    dy = torch.empty(rows, out, dtype=torch.bfloat16, device="cuda")
    for r in range(0, rows, 110000):
        dy[r:r + 110000] = rand_int(g, (110000, out), 1)
    x = rand_int(g, (rows, inn), 8).float()
    want = torch.zeros(out, inn, dtype=torch.float64, device="cuda")
    want_b = torch.zeros(out, dtype=torch.float64, device="cuda")
    for r in range(0, rows, 110000):       # exact in fp32: at most 8 x 110,000
        part = dy[r:r + 110000].float()
        want += (part.t().contiguous() @ x[r:r + 110000]).double()
        want_b += part.sum(0).double()
    w, b = wgrad(dy, pack(x, ref.INT8), inn, ref.INT8)
    assert torch.equal(w.double(), want) and torch.equal(b.double(), want_b)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dy_dt", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,out,inn", [SMALL_EXPONENTS, EXPONENTS])
def test_every_code_under_every_exponent(rows, out, inn, dy_dt, fmt):
    """dy is diagonal, so that row t of dw is 2^k times row t of the checkpoint: one product and sums with zeros,
    exact (subnormal results too)."""
    import torch
    codes = np.tile((np.arange(ref.pitch(inn)) % 256).astype(np.uint8), (rows, 1))
    if fmt == ref.E4M3:
        codes[(codes & 0x7F) == 0x7F] = 0
    top = 247 if fmt == ref.E4M3 else 249         # the last exponents that packing writes
    byte = 3 + np.arange(rows) % (top - 2)
    exps = np.tile(byte.astype(np.uint8)[:, None], (1, ref.pitch(inn) // 32))
    codes[np.abs(ref.unpack(codes, exps, ref.pitch(inn), fmt)) >= 2.0 ** 128] = 0   # not written by packing
    want = ref.unpack(codes, exps, inn, fmt)
    ck = torch.from_numpy(ref.buffer(codes, exps)).cuda()
    for k in (0, 20):
        scale = np.where(byte < 128, 2.0 ** k, 1.0)
        dy = torch.zeros(rows, out, device="cuda")
        dy[torch.arange(rows), torch.arange(rows)] = torch.from_numpy(scale.astype(np.float32)).cuda()
        w, b = wgrad(dy.bfloat16() if dy_dt == "bf16" else dy, ck, inn, fmt)
        got = w.cpu().numpy().astype(np.float64)
        exp = want * scale[:, None]
        assert np.array_equal(got[:rows], exp)
        assert not got[rows:].any() and np.array_equal(b.cpu().numpy()[:rows], scale)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dy_dt", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,out,inn", [SMALL_EXPONENTS, (700, 4097, 4100), (4000, 4300, 4100)])
def test_gradients_at_the_end_of_the_range(rows, out, inn, dy_dt, fmt):
    """dy of small multiples of 2^-133 (subnormal in bf16), x of small multiples of 2^90: exact, as the integers are."""
    import torch
    g = gen(17)
    d, x = rand_int(g, (rows, out), 4).float(), rand_int(g, (rows, inn), 8).float()
    dy = d * 2.0 ** -133
    w, b = wgrad(dy.bfloat16() if dy_dt == "bf16" else dy, pack(x * 2.0 ** 90, fmt), inn, fmt)
    assert torch.equal(w.double(), product64(d, x) * 2.0 ** -43)
    assert torch.equal(b.double(), d.double().sum(0) * 2.0 ** -133)


@pytest.mark.parametrize("fmt", FORMATS)
def test_fp32_gradients_in_three_terms(fmt):
    """fp32 dy is taken exactly down to 2^-133, the last bit that a bf16 term holds: one product per result, so one
    rounding of the whole (three terms in two sums: 2 more)."""
    import torch
    rows, out, inn = SMALL_EXPONENTS
    x = torch.ones(rows, inn, device="cuda") * 2.0 ** 20
    for e in (0, -100, -110, -111, -120, -126, -135, -149, 100):
        v = torch.rand(rows, generator=gen(e + 200), device="cuda") + 1
        v = v.double() * 2.0 ** e
        dy = torch.zeros(rows, out, device="cuda")
        at = torch.arange(rows, device="cuda")
        dy[at, at] = v.float()
        w, b = wgrad(dy, pack(x, fmt), inn, fmt)
        want = dy[at, at].double() * 2.0 ** 20
        err = (w[:rows].double() - want[:, None]).abs().max(1).values
        assert bool((err <= 3 * 2.0 ** -23 * want + (2.0 ** -113 if e < -110 else 0)).all()), e
        assert torch.equal(b[:rows], dy[at, at])


class Calls:
    """Two weight gradients in a row on one workspace, with tiles split by rows and without."""

    def __init__(self):
        import torch
        z = zr()
        self.sets = []
        for rows, out, inn, fmt in ((4000, 4300, 4100, ref.E4M3), (200000, 40, 70, ref.INT8), (700, 4097, 4100, ref.INT8)):
            e = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
            ws = torch.empty(z.zr_ckpt_wgrad_workspace_bytes(rows, out, inn), dtype=torch.uint8, device="cuda")
            self.sets.append(dict(rows=rows, out=out, inn=inn, fmt=fmt, dy=e(rows, out).bfloat16(), ws=ws,
                                  ck=torch.empty(z.zr_ckpt_bytes(rows, inn), dtype=torch.uint8, device="cuda"),
                                  dw=e(out, inn), db=e(out), dw2=e(out, inn).bfloat16(), db2=e(out).bfloat16()))

    def fill(self, seed):
        import torch
        g = gen(seed)
        for d in self.sets:
            d["dy"].copy_(torch.randn(d["dy"].shape, generator=g, device="cuda"))
            zr().zr_ckpt_pack(torch.randn(d["rows"], d["inn"], generator=g, device="cuda"), d["rows"], d["inn"], d["ck"],
                              format=d["fmt"])

    def run(self, stream=None):
        z = zr()
        for d in self.sets:
            a = (d["dy"], d["ck"], d["rows"], d["out"], d["inn"])
            k = dict(format=d["fmt"], workspace=d["ws"], stream=stream)
            z.zr_ckpt_wgrad(*a, d["dw"], dbias=d["db"], **k)
            z.zr_ckpt_wgrad(*a, d["dw2"], dbias=d["db2"], **k)
            z.zr_ckpt_wgrad(*a, d["dw"], dbias=d["db"], accumulate=True, **k)

    def equal(self, other):
        import torch
        return all(torch.equal(a[n], b[n]) for a, b in zip(self.sets, other.sets) for n in ("dw", "db", "dw2", "db2"))


def test_graph_replays_match_eager_calls():
    import torch
    g_calls, e_calls = Calls(), Calls()
    g_calls.fill(1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g_calls.run()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g_calls.run()
    for seed in range(2, 6):
        g_calls.fill(seed)
        e_calls.fill(seed)
        torch.cuda.synchronize()
        graph.replay()
        e_calls.run()
        torch.cuda.synchronize()
        assert g_calls.equal(e_calls), seed


def test_two_streams_and_results_that_do_not_change():
    import torch
    a, b, want = Calls(), Calls(), Calls()
    a.fill(1)
    b.fill(2)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for k in range(3):
        for c in (a, b):
            for d in c.sets:
                d["ws"].fill_(0xFF)       # what a workspace holds before a call does not matter
        torch.cuda.synchronize()
        a.run(stream=sa)
        b.run(stream=sb)
        torch.cuda.synchronize()
    for seed, c in ((1, a), (2, b)):
        want.fill(seed)
        want.run()
        torch.cuda.synchronize()
        assert c.equal(want)
