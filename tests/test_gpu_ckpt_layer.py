"""Norm, checkpoints and weight gradients together, as a training step has them:
the layer driver against 64 bits, through the gradient sync; captured into a
graph and replayed; and on streams of their own."""
import numpy as np
import pytest

import ckpt_ref as ref
from test_gpu_norm import backward64, forward64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def zr():
    import gradient_sync_zr_amd as m
    return m


def f64(t):
    return t.detach().cpu().double().numpy()


@pytest.mark.parametrize("fmt", [ref.E4M3, ref.INT8])
@pytest.mark.parametrize("recompute", [True, False])
def test_layer_into_the_gradient_sync(recompute, fmt):
    """K ranks' backward passes write their flat gradients from the sync's produce hook, over two micro-steps; each
    gradient is within its bound of 64 bits, and the partitions are the ring fold of the flat gradients."""
    import torch
    import oracle
    from gradient_sync_zr_amd.steps import CkptNormLinear, Zero2GradSync
    K, rows, cols, out, pad = 3, 260, 200, 136, 7
    rng = np.random.default_rng(11)
    mk = lambda *s, a=1.0: torch.from_numpy((a * rng.standard_normal(s)).astype(np.float32)).cuda()  # noqa: E731
    w, b = (1 + mk(cols, a=0.2)).bfloat16(), mk(cols, a=0.1).bfloat16()
    wl = mk(out, cols, a=0.05).bfloat16()
    flats, layers = [], []
    for r in range(K):
        flat = torch.zeros(pad + 2 * cols + out * cols + out + 5, device="cuda")
        flats.append(flat)
        layers.append(CkptNormLinear(flat, pad, rows, cols, out, format=fmt, recompute=recompute))
    assert layers[0].numel == 2 * cols + out * cols + out
    N = flats[0].numel()
    parts = [torch.empty(-(-N // K), device="cuda") for _ in range(K)]
    sync = Zero2GradSync(flats, parts, bucket=N)
    want = [np.zeros(N) for _ in range(K)]
    bound = [np.zeros(N) for _ in range(K)]
    keep = []
    for micro in range(2):
        xs = [(mk(rows, cols) + 0.2).bfloat16() for _ in range(K)]
        dzs = [mk(rows, out, a=0.01).bfloat16() for _ in range(K)]
        dxs = [mk(rows, cols, a=0.01).bfloat16() for _ in range(K)]
        olds = [d.clone() for d in dxs]
        ys = [torch.empty_like(x) for x in xs]
        dys = []
        for r in range(K):
            layers[r].forward(xs[r], w, b, ys[r])

        def produce(i, stream):
            for r in range(K):
                layers[r].backward_linear(dzs[r], accumulate=micro > 0)
                dys.append((dzs[r].float() @ wl.float()).bfloat16())
                layers[r].backward_norm(dys[r], w, dxs[r], accumulate=micro > 0, add_dx=True)

        sync.step(produce=produce)      # (a real step syncs the last micro-step only)
        torch.cuda.synchronize()
        keep.append((xs, dzs, dys))
        for r in range(K):
            hx = ref.held(f64(xs[r]), fmt)
            if recompute:               # the linear layer's input as the kernel recomputed it
                hy = ref.unpack(*ref.split(layers[r].ckpt_y.cpu().numpy(), rows, cols), cols, fmt) if r == K - 1 else None
                y64 = forward64(hx, f64(w), f64(b), 1e-5)[0]
                lay = layers[r]
                z = zr()
                z.zr_layernorm_fwd(lay.ckpt_x, rows, cols, ys[r], w, b, x_dtype=fmt)
                z.zr_ckpt_pack(ys[r], rows, cols, lay.ckpt_y, format=fmt)
                torch.cuda.synchronize()
                hy2 = ref.unpack(*ref.split(lay.ckpt_y.cpu().numpy(), rows, cols), cols, fmt)
                assert hy is None or np.array_equal(hy, hy2)
                hy = hy2
            else:
                hy = ref.unpack(*ref.split(layers[r].ckpt_y.cpu().numpy(), rows, cols), cols, fmt)
                y64 = forward64(f64(xs[r]), f64(w), f64(b), 1e-5)[0]
            # a held y is y rounded to bf16, then to the format: one step of either, and fp32's error
            step = np.abs(y64) * (2.0 ** -7 + (2.0 ** -3 if fmt == ref.E4M3 else 0)) + \
                (np.abs(y64).reshape(rows, -1)[:, :].max(1, keepdims=True) * (2.0 ** -8 if fmt == ref.E4M3 else 2.0 ** -5)) + 1e-6
            assert (np.abs(hy - y64) <= step).all()
            dz, dy = f64(dzs[r]), f64(dys[r])
            dx, dwn, dbn, bdx, bw, bb = backward64(dy, hx, f64(layers[r].mean), f64(layers[r].rstd), f64(w))
            flat = np.concatenate([dwn, dbn, (dz.T @ hy).reshape(-1), dz.sum(0)])
            mag = np.concatenate([bw, bb, (np.abs(dz).T @ np.abs(hy)).reshape(-1), np.abs(dz).sum(0)])
            want[r][pad:pad + flat.size] += flat
            bound[r][pad:pad + flat.size] += (rows + 100) * 2 * U * mag   # a sum's adds, and the two micro-steps'
            total = dx + f64(olds[r])
            lim = bdx + 2 * U * (np.abs(dx) + np.abs(f64(olds[r])))
            assert (np.abs(f64(dxs[r]) - total) <= lim + 2.0 ** -8 * (np.abs(total) + lim)).all()
    for r in range(K):
        got = f64(flats[r])
        assert (np.abs(got - want[r]) <= bound[r]).all()
    ring = oracle.reduce_scatter([f.cpu().numpy() for f in flats], N, np.float32, shift=1, average=True)
    for q in range(K):
        assert np.array_equal(parts[q].cpu().numpy().view(np.uint32), ring[q].view(np.uint32))
    sync.close()


def test_layer_arguments():
    import torch
    from gradient_sync_zr_amd.steps import CkptNormLinear
    flat = torch.zeros(1000, device="cuda")
    with pytest.raises(ValueError, match="needs"):
        CkptNormLinear(flat, 0, 16, 32, 32)
    with pytest.raises(ValueError, match="needs"):
        CkptNormLinear(flat, -1, 16, 8, 8)
    lay = CkptNormLinear(flat, 10, 16, 8, 8, bias=False)
    with pytest.raises(ValueError, match="before forward"):
        lay.backward_linear(torch.zeros(16, 8, device="cuda").bfloat16())
    with pytest.raises(ValueError, match="scratch"):
        CkptNormLinear(flat, 10, 16, 8, 8, scratch=lay.scratch[:-1])


class Step:
    """Buffers and calls of one pass through every call, two shapes of each kind."""

    def __init__(self):
        import torch
        z = zr()
        e = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
        u = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.sets = []
        for rows, cols, out, fmt in ((700, 1090, 136, ref.E4M3), (1500, 300, 77, ref.INT8), (70, 17000, 24, ref.E4M3)):
            d = dict(rows=rows, cols=cols, out=out, fmt=fmt, x=e(rows, cols).bfloat16(), dz=e(rows, out).bfloat16(),
                     dy=e(rows, cols).bfloat16(), w=e(cols), b=e(cols), y=e(rows, cols).bfloat16(),
                     y2=e(rows, cols).bfloat16(), back=e(rows, cols).bfloat16(), mean=e(rows), rstd=e(rows),
                     cx=u(z.zr_ckpt_bytes(rows, cols)), cy=u(z.zr_ckpt_bytes(rows, cols)), dx=e(rows, cols).bfloat16(),
                     dw=e(cols), db=e(cols), dl=e(out, cols), dbl=e(out),
                     ws=u(max(z.zr_layernorm_workspace_bytes(rows, cols), z.zr_ckpt_wgrad_workspace_bytes(rows, out, cols))))
            self.sets.append(d)

    OUT = ("y", "y2", "back", "mean", "rstd", "cx", "cy", "dx", "dw", "db", "dl", "dbl")

    def fill(self, seed):
        import torch
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        for d in self.sets:
            for n in ("x", "dz", "dy", "w", "b"):
                d[n].copy_(torch.randn(d[n].shape, generator=g, device="cuda"))

    def run(self, stream=None):
        z = zr()
        for d in self.sets:
            r, c, o, f = d["rows"], d["cols"], d["out"], d["fmt"]
            z.zr_layernorm_fwd(d["x"], r, c, d["y"], d["w"], d["b"], mean=d["mean"], rstd=d["rstd"], ckpt_x=d["cx"],
                               ckpt_format=f, stream=stream)
            z.zr_layernorm_fwd(d["cx"], r, c, d["y2"], d["w"], d["b"], ckpt_y=d["cy"], ckpt_format=f, x_dtype=f, stream=stream)
            z.zr_ckpt_wgrad(d["dz"], d["cy"], r, o, c, d["dl"], dbias=d["dbl"], format=f, workspace=d["ws"], stream=stream)
            z.zr_ckpt_wgrad(d["dz"], d["cy"], r, o, c, d["dl"], dbias=d["dbl"], format=f, accumulate=True, workspace=d["ws"],
                            stream=stream)
            z.zr_layernorm_bwd(d["dy"], d["cx"], r, c, d["mean"], d["rstd"], d["w"], dx=d["dx"], dweight=d["dw"],
                               dbias=d["db"], workspace=d["ws"], x_dtype=f, stream=stream)
            z.zr_layernorm_bwd(d["dy"], d["x"], r, c, d["mean"], d["rstd"], d["w"], dx=d["dx"], dweight=d["dw"],
                               dbias=d["db"], workspace=d["ws"], accumulate=True, add_dx=True, stream=stream)
            z.zr_ckpt_unpack(d["cx"], r, c, d["back"], format=f, stream=stream)
            z.zr_ckpt_pack(d["back"], r, c, d["cx"], format=f, stream=stream)

    def equal(self, other):
        import torch
        return all(torch.equal(a[n].view(torch.uint8), b[n].view(torch.uint8))
                   for a, b in zip(self.sets, other.sets) for n in self.OUT)


def test_graph_replays_match_eager_calls():
    import torch
    g_step, e_step = Step(), Step()
    g_step.fill(1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g_step.run()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g_step.run()
    for seed in range(2, 6):
        g_step.fill(seed)
        e_step.fill(seed)
        torch.cuda.synchronize()
        graph.replay()
        e_step.run()
        torch.cuda.synchronize()
        assert g_step.equal(e_step), seed


def test_streams_of_their_own():
    """Two steps at once on two streams, each with its own workspace, and calls given a stream that is not current."""
    import torch
    a, b, want = Step(), Step(), Step()
    for k, s in ((1, a), (2, b)):
        s.fill(k)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        a.run(stream=sa)
        b.run(stream=sb)
    torch.cuda.synchronize()
    for k, s in ((1, a), (2, b)):
        want.fill(k)
        want.run()
        torch.cuda.synchronize()
        assert s.equal(want)


def test_results_do_not_change_from_run_to_run():
    import torch
    a, b = Step(), Step()
    a.fill(3)
    b.fill(3)
    a.run()
    for _ in range(5):
        for d in b.sets:
            d["ws"].fill_(0xFF)       # what a workspace holds before a call does not matter
        b.run()
        torch.cuda.synchronize()
        assert a.equal(b)
