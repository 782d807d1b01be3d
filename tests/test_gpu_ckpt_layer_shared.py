"""CkptNormLinear as several layers of one rank use it: one scratch between
them, a bf16 flat gradient at odd offsets, captured and replayed, without rows,
and which statistics each half of the backward pass takes."""
import pytest

import ckpt_ref as ref

pytestmark = pytest.mark.gpu
SHAPES = [(260, 200, 136), (300, 1090, 77), (90, 4100, 24)]


def zr():
    import gradient_sync_zr_amd as m
    return m


class Rank:
    """Layers of different shapes on one flat gradient, with one scratch between them or one each."""

    def __init__(self, shared, dtype, recompute, fmt):
        import torch
        from gradient_sync_zr_amd.steps import CkptNormLinear
        numel = [2 * c + o * c + o for _, c, o in SHAPES]
        self.flat = torch.zeros(7 + sum(numel), device="cuda", dtype=dtype)
        at, scratch = 7, None
        if shared:
            sizes = [CkptNormLinear(self.flat, 7, *s, format=fmt, recompute=recompute).scratch_bytes for s in SHAPES]
            scratch = torch.empty(max(sizes), dtype=torch.uint8, device="cuda")
        self.layers, self.data = [], []
        for s, n in zip(SHAPES, numel):
            self.layers.append(CkptNormLinear(self.flat, at, *s, scratch=scratch, format=fmt, recompute=recompute))
            assert self.layers[-1].numel == n
            at += n
            e = lambda *k: torch.empty(*k, device="cuda")  # noqa: E731
            r, c, o = s
            self.data.append(dict(x=e(r, c).bfloat16(), w=e(c), b=e(c), y=e(r, c).bfloat16(), dz=e(r, o).bfloat16(),
                                  dy=e(r, c).bfloat16(), dx=e(r, c).bfloat16()))

    def fill(self, seed):
        import torch
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.flat.zero_()
        for d in self.data:
            for t in d.values():
                t.copy_(torch.randn(t.shape, generator=g, device="cuda"))

    def step(self, stream=None):
        for lay, d in zip(self.layers, self.data):
            lay.forward(d["x"], d["w"], d["b"], d["y"], stream=stream)
        for micro in (False, True):
            for lay, d in reversed(list(zip(self.layers, self.data))):
                lay.backward_linear(d["dz"], accumulate=micro, stream=stream)
                lay.backward_norm(d["dy"], d["w"], d["dx"], accumulate=micro, add_dx=micro, stream=stream)

    def same(self, other):
        import torch
        return torch.equal(self.flat, other.flat) and all(
            torch.equal(a[n], b[n]) for a, b in zip(self.data, other.data) for n in ("y", "dx"))


@pytest.mark.parametrize("recompute", [True, False])
@pytest.mark.parametrize("dtype,fmt", [("bfloat16", ref.E4M3), ("float32", ref.INT8)])
def test_layers_on_one_scratch(dtype, fmt, recompute):
    import torch
    one, each = (Rank(s, getattr(torch, dtype), recompute, fmt) for s in (True, False))
    graph_rank = Rank(True, getattr(torch, dtype), recompute, fmt)
    graph_rank.fill(1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph_rank.step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graph_rank.step()
    other = torch.cuda.Stream()
    for seed in (2, 3, 4):
        for r in (one, each, graph_rank):
            r.fill(seed)
        torch.cuda.synchronize()
        each.step()
        one.step(stream=other)      # on a stream that is not the current one
        graph.replay()
        torch.cuda.synchronize()
        assert bool(torch.isfinite(each.flat.float()).all()) and not bool(each.flat[:7].any())
        assert one.same(each) and graph_rank.same(each), seed


def test_without_rows():
    import torch
    from gradient_sync_zr_amd.steps import CkptNormLinear
    flat = torch.full((2 * 40 + 8 * 40 + 8,), 3.0, device="cuda")
    flat[5] = -0.0
    e = lambda *k: torch.empty(*k, device="cuda")  # noqa: E731
    for recompute in (True, False):
        lay = CkptNormLinear(flat, 0, 0, 40, 8, recompute=recompute)
        lay.forward(e(0, 40), e(40), e(40), e(0, 40))
        before = flat.clone()
        lay.backward_linear(e(0, 8), accumulate=True)
        lay.backward_norm(e(0, 40), e(40), e(0, 40), accumulate=True)
        torch.cuda.synchronize()
        assert torch.equal(flat.view(torch.int32), before.view(torch.int32))
    lay.backward_linear(e(0, 8))
    lay.backward_norm(e(0, 40), e(40), e(0, 40))
    torch.cuda.synchronize()
    assert not bool(flat.any())


@pytest.mark.parametrize("fmt", [ref.E4M3, ref.INT8])
def test_statistics_of_each_half(fmt):
    """backward_linear recomputes from the held values, statistics too; backward_norm takes the held values with the
    forward pass's."""
    import torch
    from gradient_sync_zr_amd.steps import CkptNormLinear
    z = zr()
    r, c, o = 70, 300, 40
    flat = torch.zeros(2 * c + o * c + o, device="cuda")
    lay = CkptNormLinear(flat, 0, r, c, o, format=fmt)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    x = (torch.randn(r, c, generator=g, device="cuda") + 3).bfloat16()
    w, b = torch.randn(c, generator=g, device="cuda"), torch.randn(c, generator=g, device="cuda")
    dy, dz = torch.randn(r, c, generator=g, device="cuda").bfloat16(), torch.randn(r, o, generator=g, device="cuda").bfloat16()
    y, dx = torch.empty_like(x), torch.empty_like(x)
    lay.forward(x, w, b, y)
    lay.backward_linear(dz)
    lay.backward_norm(dy, w, dx)
    ck = torch.empty_like(lay.ckpt_x)
    z.zr_ckpt_pack(x, r, c, ck, format=fmt)
    held = torch.empty(r, c, device="cuda")
    z.zr_ckpt_unpack(ck, r, c, held, format=fmt)
    y2, cy = torch.empty_like(x), torch.empty_like(ck)
    z.zr_layernorm_fwd(held, r, c, y2, w, b, ckpt_y=cy, ckpt_format=fmt)
    assert torch.equal(cy, lay.ckpt_y)
    m, s, d2 = torch.empty(r, device="cuda"), torch.empty(r, device="cuda"), torch.empty_like(dx)
    z.zr_layernorm_fwd(x, r, c, mean=m, rstd=s)
    z.zr_layernorm_bwd(dy, ck, r, c, m, s, w, dx=d2, x_dtype=fmt)
    assert torch.equal(d2, dx)
