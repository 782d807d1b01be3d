"""The 4-bit reference against the format's definition, by search."""
import numpy as np
import pytest

import pack_ref as pk


def test_every_code_is_its_own_nearest():
    for e in (-124, -3, 0, 120):
        x = np.concatenate([pk.TABLE, -pk.TABLE, np.zeros(16)])[None] * 2.0 ** e
        buf = pk.pack(x, pk.E2M1)
        assert buf[-1] == 127 + e
        assert np.array_equal(pk.unpack(buf, 1, 32, pk.E2M1), x)
        assert np.array_equal(np.signbit(pk.unpack(buf, 1, 32, pk.E2M1)[0, 8:16]), [True] * 8)


def test_nearest_and_error_bound():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((200, 77)) * np.exp(4 * rng.standard_normal((200, 1)))).astype(np.float32).astype(np.float64)
    h = pk.held(x, pk.E2M1)
    pad = np.zeros((200, 96))
    pad[:, :77] = np.abs(x)
    amax = pad.reshape(200, 3, 32).max(-1)
    e = np.repeat(pk.exponent(amax), 32, 1)[:, :77]
    assert (amax <= 6 * 2.0 ** pk.exponent(amax)).all() and (amax > 6 * 2.0 ** (pk.exponent(amax) - 1)).all()
    every = np.concatenate([pk.TABLE, -pk.TABLE])[:, None, None] * 2.0 ** e
    assert np.array_equal(np.abs(h - x), np.abs(every - x).min(0))
    assert (np.abs(h - x) <= np.maximum(np.abs(x) / 4, 2.0 ** (e - 2.0))).all()


@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_blocks_that_are_not_finite(bad):
    x = np.ones((2, 64))
    x[1, 40] = bad
    h = pk.held(x, pk.E2M1)
    assert np.isnan(h[1, 32:]).all() and (h[0] == 1).all() and (h[1, :32] == 1).all()


def test_top_of_the_range_stays_finite():
    x = np.full((1, 32), np.finfo(np.float32).max.astype(np.float64))
    assert pk.held(x, pk.E2M1).max() == 3 * 2.0 ** 126
