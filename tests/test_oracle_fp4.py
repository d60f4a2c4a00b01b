"""The 4-bit oracle: the code table, rounding and scales against their definitions."""
import numpy as np

from oracle import fp4 as F


def test_values():
    assert list(F.VALUES[:8]) == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert np.array_equal(F.VALUES[8:], -F.VALUES[:8])


def test_encoding_is_nearest_with_ties_to_even():
    for c in range(16):
        if c != 8:
            assert F.encode_rne(np.array([F.VALUES[c]]))[0] == c
    assert F.encode_rne(np.array([-0.0]))[0] == 8
    ties = {0.25: 0, 0.75: 2, 1.25: 2, 1.75: 4, 2.5: 4, 3.5: 6, 5.0: 6}
    for x, c in ties.items():
        assert F.encode_rne(np.array([x, -x])).tolist() == [c, c | 8]
        assert F.encode_rne(np.array([np.nextafter(x, 0)]))[0] <= c
        assert F.encode_rne(np.array([np.nextafter(x, 9)]))[0] >= c


def test_scale_is_the_smallest_that_holds_the_group():
    for amax in (1e-45, 2.0 ** -126, 6 * 2.0 ** -126, 0.3, 1.0, 1.5, 1.5000001, 6.0, 6.1, 3e38):
        k = F.scale_exp(amax)
        assert amax <= 6 * 2.0 ** k
        assert k == -126 or amax > 6 * 2.0 ** (k - 1)
    assert F.scale_exp(0.0) == 0


def test_round_trip():
    rng = np.random.default_rng(3)
    x = rng.normal(size=(5, 96)) * np.exp2(rng.integers(-9, 9, size=(5, 1)))
    x[2, 32:64] = 0
    q, s = F.quantize_groups(x)
    v = F.dequantize_groups(q, s)
    assert q.shape == (5, 48) and s.shape == (5, 3) and s[2, 1] == 127
    # half a step: 1 of the scale in the top binade (4 to 6), a quarter of it at the bottom
    step = np.repeat(np.ldexp(1.0, s.astype(int) - 127), 32, axis=1)
    assert np.all(np.abs(v - x) <= np.maximum(0.25 * step, np.abs(x) / 4))
    q2, s2 = F.quantize_groups(v)
    assert np.array_equal(F.dequantize_groups(q2, s2), v)


def test_a_group_that_is_not_finite_reads_as_nan():
    x = np.ones((2, 96))
    x[0, 40], x[1, 95] = np.inf, np.nan
    q, s = F.quantize_groups(x)
    assert s.tolist() == [[125, 255, 125], [125, 125, 255]]
    nan = np.isnan(F.dequantize_groups(q, s)).reshape(2, 3, 32)
    assert nan.all(axis=2).tolist() == nan.any(axis=2).tolist() == [[False, True, False], [False, False, True]]
