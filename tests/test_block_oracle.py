"""Pins of the float64 definitions in oracle/block_oracle.py: hand values and
identities that do not call the definition's own formula."""

import numpy as np

from oracle import block_oracle as B


def test_quant_int8_hand_values():
    # a = 2: 127 x / 2 = 127, -63.5 (tie -> even -64), 0.5 * 127 / 2 = 31.75 -> 32, 0
    q, s, total = B.quant_int8(np.array([[2.0, -1.0, 0.5, 0.0], [0.0, 0.0, 0.0, 0.0]]))
    assert q.tolist() == [[127, -64, 32, 0], [0, 0, 0, 0]]
    assert s.tolist() == [2.0 / 127.0, 1.0]
    assert total.tolist() == [95, 0]


def test_quant_int8_is_within_half_a_step():
    x = np.random.default_rng(3).standard_normal((20, 50)) * 7
    q, s, _ = B.quant_int8(x)
    assert np.abs(q * s[:, None] - x).max() <= 0.5 * s.max() * (1 + 1e-12)
    assert (np.abs(q).max(axis=1) == 127).all()


def test_unpack_int4_nibble_order():
    assert B.unpack_int4(np.array([[0x21, 0xF0]], np.uint8)).tolist() == [[1, 2, 0, 15]]


def test_w8_linear_hand_values():
    q = np.array([[1.0, 2.0], [0.0, 15.0]])
    w = np.array([[3, -1], [127, 127], [0, -128]], np.int8)
    out, acc, shift = B.w8_linear(q, [0.5, 2.0], [1.0, -4.0], w, [1.0, 0.25, 2.0], [10.0, 0.0, 0.0])
    assert acc.tolist() == [[1, 381, -256], [-15, 1905, -1920]]
    assert shift.tolist() == [[2, 254, -128], [-8, -1016, 512]]
    assert out.tolist() == [[9.5, 15.875, -128.0], [-4.0, 1460.5, -9728.0]]


def test_w8_linear_equals_dequantize_then_multiply():
    g = np.random.default_rng(5)
    q = g.integers(0, 16, (7, 40)).astype(np.float64)
    w = g.integers(-127, 128, (9, 40)).astype(np.int8)
    s, z, v = g.random(7) + 0.1, g.standard_normal(7) * 30, g.random(9) + 0.1
    out, _, _ = B.w8_linear(q, s, z, w, v, None)
    ref = (s[:, None] * (q - z[:, None])) @ (v[:, None] * w).T
    assert np.allclose(out, ref, rtol=1e-12, atol=1e-9)


def test_norms_hand_values():
    x = np.array([[3.0, 4.0, 0.0, 0.0]])  # mean square 25/4
    assert np.allclose(B.normed(x, "rms", 0.0, None, None), [[1.2, 1.6, 0.0, 0.0]])
    # mean 7/4, centred squares sum 25 - 49/4 = 51/4, variance 51/16
    sd = np.sqrt(51.0) / 4
    assert np.allclose(B.normed(x, "layer", 0.0, None, None), (x - 1.75) / sd)
    assert np.allclose(B.normed(x, "rms", 2.75, np.full(4, 2.0), np.ones(4)), [[3.0, 11.0 / 3, 1.0, 1.0]])
    assert (B.normed(x, "none", 1.0, np.full(4, 2.0), np.ones(4)) == x).all()


def test_layer_norm_ignores_shift_and_scale():
    x = np.random.default_rng(8).standard_normal((5, 64))
    assert np.allclose(B.normed(x, "layer", 0.0, None, None), B.normed(17.0 + 4.0 * x, "layer", 0.0, None, None))


def test_residual_norm_hand_values():
    h, y = np.array([[1.0, -1.0]]), np.array([[3.0, 4.0]])
    # post rms without eps: y / sqrt(12.5); gate 2, alpha 0.5 -> + y / sqrt(12.5); beta 2
    r = np.sqrt(12.5)
    hp, u = B.residual_norm(h, y, "none", "rms", 0.0, 0.0, None, None, np.array([[2.0, 2.0]]), 0.5, 2.0, None, None,
                            np.array([[1.0, 0.0]]), np.array([[0.0, 5.0]]))
    assert np.allclose(hp, [[2.0 + 3.0 / r, -2.0 + 4.0 / r]])
    assert np.allclose(u, [[2.0 * (2.0 + 3.0 / r), 3.0 + 4.0 / r]])
