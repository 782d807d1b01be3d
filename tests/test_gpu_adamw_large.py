"""AdamW on a tensor whose elements' numbers and bytes pass 32 bits in every list."""
import pytest

pytestmark = pytest.mark.gpu


def test_adamw_past_32_bits():
    """Lists off the lines by different amounts; zeros but for some elements, which become what the same elements of a small
    tensor become. All others stay as they were, those around the tensors too."""
    import torch
    import gradient_sync_zr_amd as z
    n, pad = (1 << 32) + 12345, 64
    at = torch.tensor([0, 1, 4095, (1 << 29) + 1, (1 << 30) - 1, (1 << 31) - 1, 1 << 31, (1 << 31) + 5, (1 << 32) - 1, 1 << 32,
                       (1 << 32) + 4097, n - 2, n - 1], device="cuda")
    g = torch.Generator("cuda").manual_seed(6)
    rand = lambda: torch.randn(len(at), generator=g, device="cuda")  # noqa: E731
    few = [rand().bfloat16(), rand(), rand() * 0.1, rand() ** 2, torch.empty(len(at), dtype=torch.bfloat16, device="cuda")]
    start = (7, 3, 5, 1, 2)  # of the gradients, p, m, v and the shards in their buffers
    whole, large = [], []
    for t, s in zip(few, start):
        whole.append(torch.zeros(n + pad, dtype=t.dtype, device="cuda"))
        large.append(whole[-1][s:s + n])
        if len(large) < 5:
            large[-1][at] = t
    shards = whole[4]
    shards.fill_(3.0)
    hyper = dict(step=3, lr=0.01, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
    z.zr_adamw([few[0]], [len(at)], [few[1]], [few[2]], [few[3]], shards=[few[4]], **hyper)
    z.zr_adamw([large[0]], [n], [large[1]], [large[2]], [large[3]], shards=[large[4]], **hyper)
    for small, big in zip(few, large):
        assert torch.equal(big[at], small)
    for k in range(4):
        whole[k][at + start[k]] = 0
        assert int(torch.count_nonzero(whole[k])) == 0
    large[4][at] = 0
    assert int(torch.count_nonzero(large[4])) == 0                       # p of the others, 0, in bf16
    assert bool((shards[:2] == 3).all()) and bool((shards[2 + n:] == 3).all())
