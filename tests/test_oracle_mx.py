"""Pins of the MXFP4 oracle: worked blocks, ties, the format's ends, brute force."""
import numpy as np
import pytest

from oracle import mx


def block(*head):
    b = np.zeros((1, 32))
    b[0, :len(head)] = head
    return b


def test_worked_block():
    # amax 6 -> floor(log2 6) - 2 = 0: scale 1, every level codes to itself
    c, s = mx.quantize(block(0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.5, -6.0, -0.0))
    assert s[0, 0] == 127 and list(c[0, :11]) == [0, 1, 2, 3, 4, 5, 6, 7, 9, 15, 8]


def test_ties_go_to_the_even_code():
    c, _ = mx.quantize(block(4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0))
    assert list(c[0, :8]) == [6, 0, 2, 2, 4, 4, 6, 6]


def test_saturation_and_scale_of_the_largest():
    # amax 7.9: scale 1, 7.9 saturates at 6; amax 8: scale 2, 8 = 4 * 2
    c, s = mx.quantize(block(7.9, 1.0))
    assert s[0, 0] == 127 and c[0, 0] == 7
    c, s = mx.quantize(block(8.0, 1.0))
    assert s[0, 0] == 128 and list(c[0, :2]) == [6, 1]


@pytest.mark.parametrize("amax, byte", [(0.0, 0), (2.0 ** -149, 0), (2.0 ** -126, 0), (2.0 ** -125, 0),
                                        (2.0 ** -124, 1), (1.0, 125), (3.3895313892515355e38, 252)])
def test_scale_bytes_at_the_ends(amax, byte):
    _, s = mx.quantize(block(amax))
    assert s[0, 0] == byte


def test_a_block_with_nan_or_infinity_is_nan():
    for bad in (np.nan, np.inf, -np.inf):
        x = np.concatenate([block(1.0, bad), block(1.0)], 1)
        c, s = mx.quantize(x)
        assert s[0, 0] == 255 and not c[0, :32].any() and s[0, 1] == 125
        v = mx.values(c, s)
        assert np.isnan(v[0, :32]).all() and v[0, 32] == 1.0


def test_codes_are_nearest_by_brute_force():
    g = np.random.default_rng(7)
    x = g.standard_normal((16, 96)) * np.exp2(g.integers(-20, 20, (16, 96)))
    c, s = mx.quantize(x)
    v = mx.values(c, s)
    step = np.exp2(s[:, :3].astype(float) - 127).repeat(32, 1)
    for level in np.concatenate([mx.LEVELS, -mx.LEVELS]):
        assert (np.abs(v - x) <= np.abs(level * step - x) * (1 + 1e-12)).all()
    assert (np.abs(v) <= 6 * step).all()


def test_padding():
    assert [mx.pitch(k) for k in (32, 512, 544, 1024)] == [16, 16, 32, 32]
    _, s = mx.quantize(np.ones((3, 544)))
    assert s.shape == (3, 32) and not s[:, 17:].any() and (s[:, :17] == 125).all()
