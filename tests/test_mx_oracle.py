"""The float64 definitions of the MXFP4 operators and of the per-head norms,
pinned by hand values and by brute force."""

import math

import numpy as np
import pytest

from oracle import mx_oracle as M


def test_levels_are_the_formats_values():
    # E2M1: two exponent bits with bias 1, one mantissa bit; exponent 0 is subnormal
    for code in range(8):
        e, m = code >> 1, code & 1
        assert M.LEVELS[code] == (m * 0.5 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1))


@pytest.mark.parametrize("u,code", [(0, 0), (0.25, 0), (0.2500001, 1), (0.5, 1), (0.75, 2), (1.25, 2), (1.75, 4),
                                    (2.5, 4), (2.500001, 5), (3.5, 6), (4.99, 6), (5, 6), (5.01, 7), (6, 7), (7.9, 7)])
def test_nearest_level_and_ties_to_even(u, code):
    assert M.levels_of(np.array([float(u)]))[0] == code


def test_nearest_level_by_brute_force():
    u = np.linspace(0, 8, 4001)
    got = M.LEVELS[M.levels_of(u)]
    assert np.all(np.abs(got - u)[:, None] <= np.abs(M.LEVELS[None, :] - u[:, None]) + 1e-15)


@pytest.mark.parametrize("top,floor,noclip", [(4.0, 127, 127), (6.0, 127, 127), (6.0001, 127, 128), (7.99, 127, 128),
                                              (8.0, 128, 128), (1.0, 125, 125), (2.0 ** -125, 0, 0),
                                              (2.0 ** -133, 0, 0), (0.0, 0, 0), (1.9 * 2.0 ** -125, 0, 1),
                                              (3.3e38, 252, 253)])
def test_scale_of_a_block(top, floor, noclip):
    x = np.zeros((1, 32))
    x[0, 7] = -top
    assert M.quant(x, "floor")[1][0, 0] == floor
    assert M.quant(x, "noclip")[1][0, 0] == noclip


def test_packing_padding_and_round_trip():
    x = np.zeros((2, 40))
    x[0, :4] = [6, -4, 0.5, -0.0]
    x[1, 33] = 3
    codes, scale = M.quant(x)
    assert codes.shape == (2, 32) and scale.shape == (2, 2)
    assert list(codes[0, :2]) == [7 | (14 << 4), 1 | (8 << 4)]
    assert codes[1, 16] == 7 << 4 and scale[1, 1] == 126  # 3 = 6 * 2^-1
    assert np.array_equal(M.dequant(codes, scale)[:, :40], x)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_non_finite_blocks(bad):
    x = np.ones((1, 64))
    x[0, 3] = bad
    codes, scale = M.quant(x)
    assert list(scale[0]) == [255, 125] and not codes[0, :16].any()
    y = M.dequant(codes, scale)
    assert np.isnan(y[0, :32]).all() and np.array_equal(y[0, 32:], x[0, 32:])


def test_no_value_saturates_without_clipping():
    x = np.random.default_rng(1).standard_normal((50, 320))
    for rule, most in (("floor", 8), ("noclip", 6)):
        _, scale = M.quant(x, rule)
        top = np.abs(x.reshape(50, 10, 32)).max(axis=2) / np.ldexp(1.0, scale.astype(int) - 127)
        assert top.max() <= most and top.min() > most / 2 - 1e-9


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_pairs_lengths_and_relative_angles(interleaved):
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((2, 1, 1, 8))
    angle = rng.uniform(0, 6, (1, 3))

    def turned(x, place):
        a = place * angle
        return M.qk_norm_rope(x, np.cos(a), np.sin(a), np.zeros(1, int), "none", 0.0, None, None, interleaved)[0]

    assert np.allclose((turned(q, 5) ** 2).sum(), (q ** 2).sum())
    assert np.allclose((turned(q, 5) * turned(k, 3)).sum(), (turned(q, 12) * turned(k, 10)).sum())
    assert np.array_equal(turned(q, 4)[0, 0, 6:], q[0, 0, 6:])


def test_norms_of_a_head_by_hand():
    x = np.array([[[3.0, 4.0, 0.0, 0.0]]])
    none = np.zeros((1, 0))
    at = np.zeros(1, int)
    rms, _ = M.qk_norm_rope(x, none, none, at, "rms", 0.0, np.array([1, 2, 1, 1.0]), None, False)
    assert np.allclose(rms, [[[3 / 2.5, 8 / 2.5, 0, 0]]])
    layer, _ = M.qk_norm_rope(np.array([[[1.0, 3.0]]]), none, none, at, "layer", 0.0, None, np.array([5.0, 5.0]), False)
    assert np.allclose(layer, [[[4.0, 6.0]]])
