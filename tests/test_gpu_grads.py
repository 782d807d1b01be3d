"""Gradient norm, scaling and AdamW on the GPU against their formulas in 64 bits.

Bounds, with u = 2^-24 (half a step of fp32):
 * norm, coef: squares and sums are fp64 (2^-53 each, far below u for the sizes here),
   so each is off by its one rounding: u (1 + 2^-20) of itself;
 * scaled gradients: one fp32 product, one rounding to the output: compared bit for bit
   with numpy's product and torch's cast;
 * AdamW, in roundings (every constant is one too): x = coef g 1; m: beta1 m 1, (1 - beta1) x
   with x's 3, and the sum's; v: (1 - beta2) x x with x's twice 5, beta2 v 1, the sum's 1; the
   root (v's 6, the constant and the product 2) / 2, itself 1, eps and the sum 2: 7 of itself;
   the quotient: m's own error over the root, and 8 of itself; p: the rate's constant and product 2
   more, keep p 1, the sum's 1. Results below fp32's normal range are off by a step of 2^-149 each.
"""
import numpy as np
import pytest

from gpu_util import Guarded, up16

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TINY = 2.0 ** -146  # a few steps at the bottom of fp32's range


def zr():
    import gradient_sync_zr_amd as m
    return m


def td(dt):
    import torch
    return torch.bfloat16 if dt == "bf16" else torch.float32


def bf16(a):
    """fp32 values of a rounded to bf16."""
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).bfloat16().float().numpy()


def guarded(a, dt, shift=0):
    g = Guarded(a.size, td(dt), shift)
    if a.size:
        if dt == "bf16":
            g.t.copy_(up16(np.ascontiguousarray(a, np.float32).view(np.uint32) >> 16))
        else:
            g.set(a)
    return g


def values(g):
    return g.t.float().cpu().numpy()


def make(rng, numels, dt, size=1.0):
    out = [(rng.standard_normal(n) * size * 2.0 ** (k % 5)).astype(np.float32) for k, n in enumerate(numels)]
    return [bf16(x) for x in out] if dt == "bf16" else out


def workspace(n):
    import torch
    return torch.full((max(zr().zr_grad_norm_workspace_bytes(n), 8),), 0x7F, dtype=torch.uint8, device="cuda")


def run_norm(tensors, numels, dt, **kw):
    import torch
    out = torch.full((2,), 7.0, device="cuda")
    zr().zr_grad_norm(tensors, numels, out[:1], out[1:], workspace=workspace(len(numels)),
                      dtype=zr().ZR_BF16 if dt == "bf16" else zr().ZR_FP32, **kw)
    return out.cpu().numpy().astype(np.float64)


LISTS = [[1], [3], [0, 5, 0], [16384], [16385], [4096, 4096, 4096, 4096, 1], [4095, 1, 4097, 20000, 2, 3],
         [1000003], [(k * 37) % 9000 for k in range(300)], [1] * 129, [77777, 0, 123456, 4]]


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("numels", LISTS, ids=lambda v: f"{len(v)}x{max(v)}")
def test_norm_and_scaled(numels, dt):
    rng = np.random.default_rng(len(numels) + max(numels))
    z = zr()
    for shift, scale, limit in ((0, 1.0, 1.0), (1, 1 / 3, 1e30), (29, 0.5, float("inf"))):
        xs = make(rng, numels, dt)
        gs = [guarded(x, dt, shift * (k % 3)) for k, x in enumerate(xs)]
        got = run_norm([g.ptr() for g in gs], numels, dt, scale=scale, max_norm=limit)
        norm = scale * np.sqrt(sum((x.astype(np.float64) ** 2).sum() for x in xs))
        coef = scale * min(1.0, limit / norm)
        for have, want in zip(got, (norm, coef)):
            assert abs(have - want) <= U * (1 + 2.0 ** -20) * abs(want)
        # scaled into other buffers of either type, then in place
        import torch
        k32 = np.float32(got[1])
        c = torch.full((1,), float(k32), device="cuda")
        for odt in ("bf16", "fp32"):
            outs = [Guarded(n, td(odt), (k * 5 + shift) % 67) for k, n in enumerate(numels)]
            z.zr_grad_scale([g.ptr() for g in gs], numels, c, [o.ptr() for o in outs],
                            dtype=z.ZR_BF16 if dt == "bf16" else z.ZR_FP32,
                            out_dtype=z.ZR_BF16 if odt == "bf16" else z.ZR_FP32)
            for x, o, g in zip(xs, outs, gs):
                want = x * k32
                assert np.array_equal(values(o), bf16(want) if odt == "bf16" else want)
                assert o.guards_intact() and g.guards_intact() and np.array_equal(values(g), x)
        z.zr_grad_scale([g.t for g in gs if g.n], [n for n in numels if n], c)
        for x, g in zip(xs, gs):
            want = x * k32
            assert np.array_equal(values(g), bf16(want) if dt == "bf16" else want) and g.guards_intact()


def test_norm_range_and_values_that_are_not_finite():
    """Squares that fp32 does not hold; a NaN or an infinity anywhere gives a NaN coefficient; zeros are not clipped."""
    import torch
    z = zr()
    for dt in ("bf16", "fp32"):
        for n in (5, 100000):
            for v in (1e-30, 2.0 ** -140 if dt == "fp32" else 2.0 ** -126, 1e30, 3e38):
                x = np.full(n, v, np.float32)
                x = bf16(x) if dt == "bf16" else x
                norm = float(x[0]) * np.sqrt(n)
                with np.errstate(over="ignore"):
                    want = float(np.float32(norm))
                got = run_norm([guarded(x, dt).t], [n], dt, max_norm=1.0)
                if np.isinf(want):  # the norm passes fp32's range, the coefficient does not
                    assert np.isinf(got[0])
                else:
                    assert abs(got[0] - want) <= 2 * U * want + TINY
                assert abs(got[1] - min(1.0, 1.0 / norm)) <= 2 * U * min(1.0, 1.0 / norm) + TINY
            for bad in (np.nan, np.inf, -np.inf):
                for where in (0, n // 2, n - 1):
                    x = np.ones(n, np.float32)
                    x[where] = bad
                    got = run_norm([guarded(np.ones(3, np.float32), dt).t, guarded(x, dt).t], [3, n], dt, max_norm=1.0)
                    assert not np.isfinite(got[0]) and np.isnan(got[1])
            got = run_norm([torch.zeros(n, device="cuda", dtype=td(dt))], [n], dt, max_norm=1e-3, scale=0.25)
            assert got[0] == 0.0 and got[1] == 0.25
    assert list(run_norm([], [], "fp32", scale=0.5)) == [0.0, 0.5]
    # a NaN coefficient marks every element; 1 leaves the gradients' bits (a signalling NaN's too) as they are
    x = torch.tensor([0x7F800001, 0x3F800000, -0x80000000], dtype=torch.int64).to(torch.int32).cuda().view(torch.float32)
    keep = x.view(torch.int32).clone()
    z.zr_grad_scale([x], [3], torch.ones(1, device="cuda"))
    assert torch.equal(x.view(torch.int32), keep)
    z.zr_grad_scale([x], [3], torch.full((1,), float("nan"), device="cuda"))
    assert bool(torch.isnan(x).all())


def test_norm_past_32_bits():
    """An element count and byte offsets past 2^32."""
    import torch
    n = (1 << 32) + 12345
    x = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    x[0], x[(1 << 31) + 5], x[-1] = 3.0, 4.0, 12.0
    got = run_norm([x], [n], "bf16", max_norm=6.5)
    assert got[0] == 13.0 and got[1] == 0.5
    c = torch.full((1,), 0.5, device="cuda")
    zr().zr_grad_scale([x], [n], c)
    assert [float(x[i]) for i in (0, (1 << 31) + 5, n - 1)] == [1.5, 2.0, 6.0] and int((x != 0).sum()) == 3


# ------------------------------------------------------------------ AdamW
def adam64(g, p, m, v, coef, lr, b1, b2, eps, wd, step):
    """New p, m, v and their bounds."""
    x = coef * g
    m1 = b1 * m + (1 - b1) * x
    bm = U * (2 * np.abs(b1 * m) + 3 * np.abs((1 - b1) * x) + np.abs(m1)) + TINY
    v1 = b2 * v + (1 - b2) * x * x
    bv = U * (2 * b2 * v + 6 * (1 - b2) * x * x + v1) + TINY
    root = np.sqrt(v1 / (1 - b2 ** step)) + eps
    low = np.maximum(root * (1 - 8 * U) - np.sqrt(TINY / (1 - b2 ** step)), 1e-300)
    rate = lr / (1 - b1 ** step)
    q = m1 / root
    off = np.abs(m1) * (1 / low - 1 / root) + bm / low + 8 * U * np.abs(q)
    p1 = (1 - lr * wd) * p - rate * q
    bp = U * (2 * np.abs(p) + np.abs(p1)) + rate * off + 3 * U * rate * np.abs(q) + TINY
    return (p1, m1, v1), (bp, bm, bv)


def state(rng, numels, dt, shift):
    g = make(rng, numels, dt, 1e-3)
    p, m = make(rng, numels, "fp32", 0.02), make(rng, numels, "fp32", 1e-4)
    v = [x * x for x in make(rng, numels, "fp32", 1e-3)]
    bufs = [[guarded(x, d, shift * (j * 7 + k * 5) % 67) for k, x in enumerate(xs)]
            for j, (xs, d) in enumerate(((g, dt), (p, "fp32"), (m, "fp32"), (v, "fp32")))]
    shards = [Guarded(n, td("bf16"), shift * (k * 3 + 1) % 67) for k, n in enumerate(numels)]
    return (g, p, m, v), bufs, shards


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("numels", LISTS, ids=lambda v: f"{len(v)}x{max(v)}")
def test_adamw(numels, dt):
    import torch
    z = zr()
    rng = np.random.default_rng(len(numels) * 3 + max(numels))
    for shift, coef, hyper in ((0, None, dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, step=1)),
                               (1, 0.37, dict(lr=0.02, beta1=0.0, beta2=0.95, eps=1e-6, weight_decay=0.0, step=12345)),
                               (3, 1.0, dict(lr=3e-4, beta1=0.95, beta2=0.0, eps=1e-10, weight_decay=0.5, step=2))):
        host, bufs, shards = state(rng, numels, dt, shift)
        c = None if coef is None else torch.full((1,), coef, device="cuda")
        k = 1.0 if coef is None else float(np.float32(coef))
        ptrs = [[b.ptr() for b in bs] for bs in bufs]
        z.zr_adamw(ptrs[0], numels, *ptrs[1:], shards=None if shift == 3 else [s.ptr() for s in shards], coef=c,
                   dtype=z.ZR_BF16 if dt == "bf16" else z.ZR_FP32, **hyper)
        names = {"lr": "lr", "beta1": "b1", "beta2": "b2", "eps": "eps", "weight_decay": "wd", "step": "step"}
        for i in range(len(numels)):
            want, bound = adam64(*(x[i].astype(np.float64) for x in host), k, **{names[n]: a for n, a in hyper.items()})
            for j in range(3):
                got = values(bufs[j + 1][i]).astype(np.float64)
                assert (np.abs(got - want[j]) <= bound[j]).all(), (i, j)
            assert np.array_equal(values(bufs[0][i]), host[0][i])
            if shift != 3:
                assert np.array_equal(values(shards[i]), bf16(values(bufs[1][i])))
            else:
                assert bool((shards[i].t.view(torch.int16) == -1).all())
            assert all(bs[i].guards_intact() for bs in bufs) and shards[i].guards_intact()


def test_adamw_left_out_where_the_coefficient_is_not_finite():
    import torch
    z = zr()
    rng = np.random.default_rng(3)
    numels = [100, 5000]
    for bad in (float("nan"), float("inf"), float("-inf")):
        host, bufs, shards = state(rng, numels, "fp32", 1)
        z.zr_adamw([b.ptr() for b in bufs[0]], numels, *([b.ptr() for b in bs] for bs in bufs[1:]), step=1, lr=0.1,
                   shards=[s.ptr() for s in shards], coef=torch.full((1,), bad, device="cuda"), dtype=z.ZR_FP32)
        for xs, bs in zip(host, bufs):
            assert all(np.array_equal(values(b), x) for x, b in zip(xs, bs))
        assert all(bool((s.t.view(torch.int16) == -1).all()) for s in shards)


def test_adamw_values_that_are_not_finite_stay_where_they_are():
    """Without a coefficient a NaN gradient reaches its own element alone."""
    import torch
    z = zr()
    g = torch.ones(9000, device="cuda")
    g[4097], g[8999] = float("nan"), float("inf")
    p, m, v = (torch.zeros(9000, device="cuda") for _ in range(3))
    z.zr_adamw([g], [9000], [p], [m], [v], step=1, lr=0.1, weight_decay=0.0)
    bad = [4097, 8999]
    assert not bool(torch.isfinite(p[bad]).any())
    p[bad] = float(p[0])
    assert bool((p == p[0]).all()) and abs(float(p[0]) + 0.1) < 1e-6


# ---------------------------------------------------- together, and streams
def one_step(z, grads, numels, out, ws, p, m, v, shards):
    z.zr_grad_norm(grads, numels, out[:1], out[1:], max_norm=1.0, workspace=ws)
    z.zr_adamw(grads, numels, p, m, v, step=3, lr=0.01, shards=shards, coef=out[1:])


def test_captured_and_replayed_with_tables():
    """Norm, scaling and AdamW in one graph over prepared tables, replayed on new gradients, equal the eager calls."""
    import torch
    z = zr()
    numels = [70001, 3, 0, 4096, 20000]
    new = lambda seed: [torch.randn(n, device="cuda", generator=torch.Generator("cuda").manual_seed(seed + i))  # noqa: E731
                        for i, n in enumerate(numels)]
    g, scaled = new(1), [torch.empty(n, dtype=torch.bfloat16, device="cuda") for n in numels]
    p, m = new(50), new(60)
    v = [x * x for x in new(70)]
    out, ws = torch.zeros(2, device="cuda"), workspace(len(numels))
    tables = [z.tensor_table(x, numels) for x in (g, p, m, v, scaled)]

    def calls():
        z.zr_grad_norm(tables[0], numels, out[:1], out[1:], max_norm=1.0, workspace=ws)
        z.zr_grad_scale(tables[0], numels, out[1:], tables[4])
        z.zr_adamw(*tables[:1], numels, *tables[1:4], step=3, lr=0.01, coef=out[1:])

    start = [[x.clone() for x in xs] for xs in (p, m, v)]
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        calls()
    for seed in (100, 200, 300):
        fresh = new(seed)
        sides = []
        for how in ("eager", "replay"):
            for x, y in zip(g, fresh):
                x.copy_(y)
            for xs, ys in zip((p, m, v), start):
                for x, y in zip(xs, ys):
                    x.copy_(y)
            out.zero_()
            calls() if how == "eager" else graph.replay()
            torch.cuda.synchronize()
            sides.append([t.clone() for xs in ([out], p, m, v, scaled) for t in xs])
        assert all(torch.equal(a, b) for a, b in zip(*sides))
        assert float(out[0]) > 1.0


def test_on_another_stream():
    import torch
    z = zr()
    numels = [300000, 17]
    g = [torch.randn(n, device="cuda") for n in numels]
    state = [[torch.rand(n, device="cuda") for n in numels] for _ in range(3)]
    sh = [torch.empty(n, dtype=torch.bfloat16, device="cuda") for n in numels]
    sides = []
    for k in range(2):
        p, m, v = ([x.clone() for x in xs] for xs in state)
        out, ws = torch.zeros(2, device="cuda"), workspace(2)
        s = torch.cuda.Stream() if k else torch.cuda.current_stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            one_step(z, g, numels, out, ws, p, m, v, sh)
        torch.cuda.current_stream().wait_stream(s)
        sides.append([t.clone() for xs in ([out], p, m, v, sh) for t in xs])
        torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*sides))


def test_the_same_gradient_twice_and_runs_alike():
    import torch
    z = zr()
    x = torch.randn(500000, device="cuda")
    a = run_norm([x, x], [500000] * 2, "fp32")
    b = run_norm([x], [500000], "fp32")
    assert abs(a[0] - np.sqrt(2) * b[0]) <= 4 * U * a[0]
    assert all((run_norm([x, x], [500000] * 2, "fp32") == a).all() for _ in range(5))


def test_arguments_on_the_gpu_are_checked():
    import torch
    z = zr()
    g = [torch.zeros(10, device="cuda"), torch.zeros(5, device="cuda", dtype=torch.bfloat16)]
    out = torch.zeros(2, device="cuda")
    with pytest.raises(ValueError, match="among others"):
        z.zr_grad_norm(g, [10, 5], out[:1], workspace=workspace(2))
    with pytest.raises(ValueError, match="not 9 contiguous"):
        z.zr_grad_norm(g[:1], [9], out[:1], workspace=workspace(1))
    with pytest.raises(ValueError, match="contiguous"):
        z.zr_grad_norm([torch.zeros(10, 2, device="cuda")[:, 0]], [10], out[:1], workspace=workspace(1))
    with pytest.raises(ValueError, match="norm is not 1"):
        z.zr_grad_norm(g[:1], [10], out, workspace=workspace(1))
    with pytest.raises(ValueError, match="dtype"):
        z.zr_adamw(g[:1], [10], g[:1], g[1:], g[:1], step=1, lr=0.1)
