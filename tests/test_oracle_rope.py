"""The rotary oracle against complex multiplication, and its group property."""

import numpy as np
import pytest

from oracle.rope import angle_table, rotate32, rotate64


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot,d", [(2, 2), (6, 8), (64, 64), (32, 128)])
def test_rotation_is_complex_multiplication(rot, d, interleaved):
    rng = np.random.default_rng(rot + d)
    x = rng.standard_normal((5, 3, d))
    ang = rng.uniform(-np.pi, np.pi, (5, rot // 2))
    y = rotate64(x, np.concatenate([np.cos(ang), np.sin(ang)], 1), interleaved)
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * ang)[:, None]
    # three roundings of values up to |z|, in float64
    assert np.max(np.abs(y[..., a] - z.real)) <= 8 * np.finfo(np.float64).eps * np.max(np.abs(z))
    assert np.max(np.abs(y[..., b] - z.imag)) <= 8 * np.finfo(np.float64).eps * np.max(np.abs(z))
    assert np.array_equal(y[..., rot:], x[..., rot:])


def test_scores_depend_on_the_distance_alone():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 1, 64))
    t = angle_table(64, 64).astype(np.float64)
    dots = [float((rotate64(q, t[p + 7:p + 8], False) * rotate64(k, t[p:p + 1], False)).sum()) for p in (0, 11, 50)]
    # the table is float32: its entries are off by 2^-25 each, two tables, 64 products up to |q||k|
    assert np.ptp(dots) <= 64 * 4 * 2.0 ** -24 * np.max(np.abs(q)) * np.max(np.abs(k))


def test_position_zero_is_the_identity_and_float32_is_near():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((4, 2, 16)).astype(np.float32)
    t = angle_table(9, 16)
    assert np.array_equal(rotate32(x, t[:1].repeat(4, 0), False), x)
    rows = t[[1, 3, 8, 5]]
    # two products and a sum, half a step each of at most |a c| + |b s| <= 2 max|x|
    assert np.max(np.abs(rotate32(x, rows, True) - rotate64(x, rows, True))) <= 2 * 2 * 2.0 ** -24 * np.max(np.abs(x))
