"""The 64-bit reference of the 8-bit checkpoint format against hand-derived values."""
import numpy as np
import pytest

import ckpt_ref as ref


def test_tables():
    t = ref.table(ref.E4M3)
    assert t.size == 127 and t[0] == 0 and t[1] == 2.0 ** -9 and t[8] == 2.0 ** -6 and t[126] == 448
    assert (np.diff(t) > 0).all()


@pytest.mark.parametrize("fmt", [ref.E4M3, ref.INT8])
def test_exponent_at_its_borders(fmt):
    top = ref.TOP[fmt]
    for k in (-100, -7, 0, 5, 100):
        assert ref.exponent(np.array(top * 2.0 ** k), fmt) == k
        assert ref.exponent(np.nextafter(np.float32(top * 2.0 ** k), np.float32(np.inf)).astype(np.float64), fmt) == k + 1
    assert ref.exponent(np.array(0.0), fmt) == -124
    assert ref.exponent(np.array(2.0 ** -140), fmt) == -124


def test_hand_derived_blocks():
    x = np.zeros((1, 32))
    x[0, :6] = [448, 18, 19, -20, 2.0 ** -10, 3 * 2.0 ** -10]   # e = 0; 19 is between 18 and 20, 18's code is odd
    codes, exps = ref.pack(x, ref.E4M3)
    assert exps[0, 0] == 127
    t = ref.table(ref.E4M3)
    got = ref.unpack(codes, exps, 32, ref.E4M3)[0, :6]
    assert list(got) == [448, 18, 20, -20, 0, 2.0 ** -8]      # ties: to even codes, 2^-10 to 0, 3 * 2^-10 to 2^-8
    assert t[codes[0, 0]] == 448
    x[0, :6] = [127, 0.5, 1.5, -2.5, -127, 126.5]
    codes, exps = ref.pack(x, ref.INT8)
    assert exps[0, 0] == 127 and list(codes[0, :6]) == [127, 0, 2, 254, 129, 126]


def test_blocks_that_are_not_finite_and_the_largest():
    x = np.ones((2, 40))
    x[0, 3] = np.inf
    x[1, 35] = np.nan
    for fmt in (ref.E4M3, ref.INT8):
        got = ref.held(x, fmt)
        assert np.isnan(got[0, :32]).all() and np.isfinite(got[0, 32:]).all()
        assert np.isfinite(got[1, :32]).all() and np.isnan(got[1, 32:]).all()
    big = np.full((1, 32), float(np.finfo(np.float32).max))
    assert ref.held(big, ref.E4M3)[0, 0] == 1.875 * 2.0 ** 127
    assert ref.held(big, ref.INT8)[0, 0] == 63 * 2.0 ** 122


@pytest.mark.parametrize("fmt", [ref.E4M3, ref.INT8])
def test_error_bound_and_bf16(fmt):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((64, 96)) * np.exp(rng.standard_normal((64, 96)))
    h = ref.held(x, fmt)
    e = ref.exponent(np.abs(x.reshape(64, 3, 32)).max(-1), fmt).repeat(32, 1).astype(np.float64)
    bound = np.maximum(2.0 ** -4 * np.abs(x), np.exp2(e - 10)) if fmt == ref.E4M3 else np.exp2(e - 1)
    assert (np.abs(h - x) <= bound).all()
    bits = h.astype(np.float32).view(np.uint32)
    assert (h.astype(np.float32) == h).all() and (bits & 0xFFFF == 0).all()   # exact in bf16
