"""CPU pins of the key/value cache oracle: the quantiser against a search over
every e4m3 value, its scale's definition, and the attention masks."""
import numpy as np
import pytest

from oracle import fp8, kv


def e4m3_values():
    return np.unique(fp8.TABLE[np.isfinite(fp8.TABLE)])


def test_rounding_is_to_the_nearest_value_ties_to_even():
    vals = e4m3_values()
    rng = np.random.default_rng(3)
    mids = (vals[1:] + vals[:-1]) / 2
    x = np.concatenate([vals, mids, rng.uniform(-448, 448, 2000), rng.normal(0, 0.01, 2000)])
    got = kv.e4m3_round(x)
    assert np.isin(got, vals).all()
    best = np.abs(x[:, None] - vals[None, :]).min(1)
    assert (np.abs(got - x) == best).all()
    # a tie goes to the value whose last significant bit is zero
    _, e = np.frexp(np.maximum(np.abs(kv.e4m3_round(mids)), 2.0 ** -6))
    assert (np.mod(kv.e4m3_round(mids) / np.ldexp(1.0, e - 4), 2) == 0).all()


@pytest.mark.parametrize("amax", [0.0, 448.0, 448.0000001, 449.0, 1.0, 0.875, 0.8750001, 2.0 ** -126, 3.0e38, 447.9])
def test_scale_is_the_smallest_power_that_holds_the_vector(amax):
    k = kv.scale_exponent(amax)
    assert amax <= 448.0 * 2.0 ** k and k >= -110
    assert k == -110 or amax > 448.0 * 2.0 ** (k - 1)


def test_quantised_vectors_read_back_as_finite_bf16_values_or_nan():
    big = float(np.uint32(0x7f7f0000).view(np.float32))  # the largest bf16 value
    x = np.array([[big, -big, 1.0, 0.0], [np.inf, 1.0, 2.0, 3.0], [np.nan, 1.0, 2.0, 3.0], [0.0] * 4, [1e-30] * 4])
    codes, e = kv.quantise(x)
    y = kv.dequantise(codes, e)
    assert e.tolist() == [247, 255, 255, 17, 19]
    assert np.isnan(y[1:3]).all() and np.isfinite(y[[0, 3, 4]]).all()
    f32 = y[[0, 3, 4]].astype(np.float32)
    assert (f32.astype(np.float64) == y[[0, 3, 4]]).all() and not (f32.view(np.uint32) & 0xffff).any()
    assert y[0, 0] == 240.0 * 2.0 ** 120


def test_masks():
    assert kv.visible(4, 2, True, 0).tolist() == [[True, True, True, False], [True] * 4]
    assert kv.visible(4, 2, True, 2).tolist() == [[False, True, True, False], [False, False, True, True]]
    assert kv.visible(2, 3, True, 0).tolist() == [[False, False], [True, False], [True, True]]  # position -1 sees nothing
    out, lse, _, _ = kv.attend(np.ones((3, 1, 4)), np.ones((2, 1, 4)), np.ones((2, 1, 4)), 0.5)
    assert (out[0] == 0).all() and np.isneginf(lse[0]).all() and np.allclose(out[1:], 1)


def test_a_negative_position_sees_nothing_without_the_causal_mask():
    assert kv.visible(2, 3, False, 0).tolist() == [[False, False], [True, True], [True, True]]
    assert kv.visible(0, 2, False, 0).shape == (2, 0) and kv.visible(3, 2, False, 0).all()
