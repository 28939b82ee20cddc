"""Plain float64 definitions of the 8-bit products, the INT8 quantizer and the
norms around a block (numpy; used by tests only)."""

import numpy as np


def quant_int8(x):
    """x float64 [T, n] -> (codes, scale, sum): a = max|x|, codes = rint(127 x / a)
    (ties to even), scale = a / 127, both for a > 0; codes 0 and scale 1 else."""
    x = np.asarray(x, np.float64)
    a = np.abs(x).max(axis=1, keepdims=True)
    some = a > 0
    q = np.rint(127.0 * x / np.where(some, a, 1.0)) * some
    scale = np.where(some, a / 127.0, 1.0)[:, 0]
    return q.astype(np.int8), scale, q.sum(axis=1).astype(np.int32)


def unpack_int4(codes):
    """u8 [T, n/2] -> [T, n]: channel 2m in the low nibble of byte m."""
    out = np.empty((codes.shape[0], 2 * codes.shape[1]), np.float64)
    out[:, 0::2] = codes & 15
    out[:, 1::2] = codes >> 4
    return out


def w8_linear(q, scale, zero, w, w_scale, bias):
    """s v (q . w - z sum w) + b with q float64 [T, n] whole numbers, zero None
    for symmetric codes.  Returns (out, whole sums q . w, z sum w)."""
    w = np.asarray(w, np.float64)
    acc = q @ w.T
    shift = np.zeros_like(acc) if zero is None else np.outer(np.asarray(zero, np.float64), w.sum(axis=1))
    out = np.asarray(scale, np.float64)[:, None] * np.asarray(w_scale, np.float64)[None, :] * (acc - shift)
    if bias is not None:
        out = out + np.asarray(bias, np.float64)[None, :]
    return out, acc, shift


def norm_parts(x, kind, eps):
    """(mean, 1 / sqrt(var + eps)) per row; (0, 1) for "none"."""
    if kind == "none":
        return np.zeros((x.shape[0], 1)), np.ones((x.shape[0], 1))
    mean = x.mean(axis=1, keepdims=True) if kind == "layer" else np.zeros((x.shape[0], 1))
    return mean, 1.0 / np.sqrt(((x - mean) ** 2).mean(axis=1, keepdims=True) + eps)


def normed(x, kind, eps, weight, bias):
    mean, inv = norm_parts(x, kind, eps)
    if kind == "none":
        return x
    v = (x - mean) * inv
    v = v if weight is None else v * weight
    return v if bias is None else v + bias


def residual_norm(h, y, norm, post_norm, eps, post_eps, post_weight, post_bias, gate, alpha, beta, weight, bias,
                  mod_scale, mod_shift):
    """(h', u); gate, mod_scale and mod_shift already spread to [T, n] or [1, n]."""
    hp = beta * h
    if y is not None:
        b = normed(y, post_norm, post_eps, post_weight, post_bias)
        hp = hp + alpha * (b if gate is None else gate * b)
    u = normed(hp, norm, eps, weight, bias)
    if mod_scale is not None:
        u = u * (1.0 + mod_scale)
    if mod_shift is not None:
        u = u + mod_shift
    return hp, u
