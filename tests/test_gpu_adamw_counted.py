"""AdamW where steps are left out: the corrections go by the updates that were made."""
import numpy as np
import pytest

from test_gpu_grads import adam64, guarded, make, values

pytestmark = pytest.mark.gpu

HYPER = dict(lr=0.01, b1=0.9, b2=0.95, eps=1e-8, wd=0.1)


def test_clipped_steps_of_gradients_that_are_not_finite():
    """Bad steps first and in between: every good one is the formula's, numbered among the good ones; the bad leave all as
    it was and are counted once, also where the lists take several launches."""
    import torch
    from gradient_sync_zr_amd.steps import ClipAdamW
    rng = np.random.default_rng(8)
    numels = [300 + k % 7 for k in range(130)]
    lists = [make(rng, numels, "fp32", size) for size in (1e-3, 0.02, 0.0, 0.0)]
    g, p, m, v = ([torch.from_numpy(x).cuda() for x in xs] for xs in lists)
    shards = [x.bfloat16() for x in p]
    opt = ClipAdamW(g, p, m, v, shards, lr=0.01, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, max_norm=0.3, scale=0.5)
    made = 0
    for k, bad in enumerate((float("nan"), float("inf"), 0.0, 0.0, float("nan"), 0.0)):
        for x, fresh in zip(g, make(rng, numels, "fp32", 1e-3)):
            x.copy_(torch.from_numpy(fresh))
        if bad:
            g[77][5] = bad
        before = [[x.double().cpu().numpy() for x in xs] for xs in (g, p, m, v)]
        keep = [x.clone() for xs in (p, m, v, shards) for x in xs]
        opt.step()
        made += not bad
        assert opt.steps == k + 1 and int(opt.left_out) == k + 1 - made
        if bad:
            assert all(torch.equal(a, b) for a, b in zip(keep, [x for xs in (p, m, v, shards) for x in xs]))
            continue
        coef = float(opt.coef)
        for i in range(len(numels)):
            want, lim = adam64(*(b[i] for b in before), coef, step=made, **HYPER)
            for got, w, bound in zip((p[i], m[i], v[i]), want, lim):
                assert (np.abs(got.double().cpu().numpy() - w) <= bound).all(), (k, i)
            assert torch.equal(shards[i], p[i].bfloat16())


def test_counted_and_plain():
    """Without a step left out the bits are zr_adamw's; with some, those of the smaller number to a rounding of the
    corrections; never below the first."""
    import torch
    import gradient_sync_zr_amd as z
    rng = np.random.default_rng(2)
    numels = [5000, 1, 4097]
    host = [make(rng, numels, "fp32", size) for size in (1e-3, 0.02, 1e-4, 1e-3)]
    host[3] = [x * x for x in host[3]]

    def run(step, left=None):
        bufs = [[guarded(x, "fp32", 1) for x in xs] for xs in host]
        count = None if left is None else torch.tensor([left], device="cuda")
        z.zr_adamw(*([b.ptr() for b in bs] for bs in bufs[:1]), numels, *([b.ptr() for b in bs] for bs in bufs[1:]), step=step,
                   lr=0.01, beta1=0.9, beta2=0.95, weight_decay=0.1, dtype=z.ZR_FP32, left_out=count)
        assert count is None or int(count) == left
        assert all(b.guards_intact() for bs in bufs for b in bs)
        return [[values(b) for b in bs] for bs in bufs[1:]]

    same = lambda a, b: all(np.array_equal(x, y) for xs, ys in zip(a, b) for x, y in zip(xs, ys))  # noqa: E731
    assert same(run(7, 0), run(7))
    for step, left, number in ((12, 5, 7), (1000003, 1000000, 3), (4, 4, 1), (2, 9, 1), ((1 << 40) + 2, 1 << 40, 2), (5000, 1, 4999)):
        got = run(step, left)
        for i in range(len(numels)):
            want, lim = adam64(*(x[i].astype(np.float64) for x in host), 1.0, step=number, **HYPER)
            for j in range(3):
                assert (np.abs(got[j][i].astype(np.float64) - want[j]) <= lim[j]).all(), (step, left, i, j)


def test_types_are_checked_when_the_step_is_made():
    """Not behind its first norm."""
    import torch
    from gradient_sync_zr_amd.steps import ClipAdamW
    f, b = (torch.zeros(8, dtype=dt, device="cuda") for dt in (torch.float32, torch.bfloat16))
    ClipAdamW([b], [f], [f.clone()], [f.clone()], [b.clone()])
    for bad in ([[f], [b], [f], [f]], [[f], [f], [b], [f]], [[f], [f], [f], [b]], [[f], [f], [f], [f], [f]]):
        with pytest.raises(ValueError, match="dtype"):
            ClipAdamW(*bad)


def test_first_step_on_another_stream():
    """The count of steps left out is there before the constructor returns, whatever the current stream has in front."""
    import torch
    from gradient_sync_zr_amd.steps import ClipAdamW
    sides = []
    for busy in (False, True):
        g, p, m, v = (torch.full((5000,), x, device="cuda") for x in (0.5, 1.0, 0.0, 0.0))
        old = torch.full((1,), 1 << 40, device="cuda")  # what the count's memory may hold
        a = torch.ones(4096, 4096, device="cuda")
        stream = torch.cuda.Stream()
        torch.cuda.synchronize()
        if busy:
            for _ in range(20):
                a = a @ a * 1e-4
        del old
        opt = ClipAdamW([g], [p], [m], [v], lr=0.1)
        opt.steps = 6
        with torch.cuda.stream(stream):
            opt.step()
        torch.cuda.synchronize()
        assert int(opt.left_out) == 0 and opt.steps == 7
        sides.append([p, m, v])
    assert all(torch.equal(x, y) for x, y in zip(*sides))
