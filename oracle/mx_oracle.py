"""Plain float64 definitions of the MXFP4 quantizer and product and of the
per-head norms with the position rotation (numpy; used by tests only)."""

import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def levels_of(u):
    """Codes (0..7) of magnitudes u >= 0: the nearest level, the even code at a tie."""
    codes = np.zeros(u.shape, np.uint8)
    for c in range(1, 8):
        half = (LEVELS[c - 1] + LEVELS[c]) / 2
        codes[(u >= half) if c % 2 == 0 else (u > half)] = c
    return codes


def quant(x, rule="floor"):
    """x float64 [T, n] -> (codes u8 [T, 16 nb], scale bytes u8 [T, nb])."""
    x = np.asarray(x, np.float64)
    t, n = x.shape
    nb = (n + 31) // 32
    b = np.zeros((t, 32 * nb))
    b[:, :n] = x
    b = b.reshape(t, nb, 32)
    top = np.abs(b).max(axis=2)  # NaN stays
    good = np.isfinite(top)
    safe = np.where(good & (top > 0), top, 1.0)
    e = np.frexp(safe)[1] - 1 - 2
    if rule == "noclip":
        e = e + (safe > 6.0 * np.ldexp(1.0, e))
    e = np.clip(np.where(top > 0, e, -127), -127, 127)
    codes = levels_of(np.where(good[:, :, None], np.abs(b), 0.0) / np.ldexp(1.0, e)[:, :, None])
    codes |= (np.signbit(b).astype(np.uint8) << 3)
    codes[~good] = 0
    packed = codes[:, :, 0::2] | (codes[:, :, 1::2] << 4)
    return packed.reshape(t, 16 * nb), np.where(good, e + 127, 255).astype(np.uint8)


def dequant(codes, scale):
    """float64 [T, 32 nb] of codes and scale bytes."""
    c = np.empty((codes.shape[0], 2 * codes.shape[1]), np.uint8)
    c[:, 0::2] = codes & 15
    c[:, 1::2] = codes >> 4
    v = np.where(c & 8, -LEVELS[c & 7], LEVELS[c & 7])
    s = np.where(scale == 255, np.nan, np.ldexp(1.0, scale.astype(np.int64) - 127))
    return v * np.repeat(s, 32, axis=1)


def linear(x, w, bias=None):
    """(x w^T + b, |x| |w|^T): the product and the sum of its terms' magnitudes."""
    out, size = x @ w.T, np.abs(x) @ np.abs(w).T
    return (out if bias is None else out + np.asarray(bias, np.float64)), size


def qk_norm_rope(x, cos, sin, places, norm, eps, weight, bias, interleaved):
    """x float64 [T, H, D]; cos and sin [P, R] float64 read at row places[t] ->
    (result, normed x)."""
    v = x
    if norm != "none":
        if norm == "layer":
            v = v - v.mean(axis=2, keepdims=True)
        v = v / np.sqrt((v * v).mean(axis=2, keepdims=True) + eps)
        if weight is not None:
            v = v * weight
        if bias is not None:
            v = v + bias
    out = v.copy()
    r = cos.shape[1]
    c, s = cos[places][:, None, :], sin[places][:, None, :]
    a, b = (slice(0, 2 * r, 2), slice(1, 2 * r, 2)) if interleaved else (slice(0, r), slice(r, 2 * r))
    out[:, :, a] = v[:, :, a] * c - v[:, :, b] * s
    out[:, :, b] = v[:, :, b] * c + v[:, :, a] * s
    return out, v
