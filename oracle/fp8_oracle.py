"""fp64 CPU oracle for 8-bit rows and weights with block scales, and for the gated feed-forward block.

TEST INFRASTRUCTURE ONLY, like gq_oracle: NumPy, float64, plain definitions.

A code is e4m3: sign, four exponent bits (bias 7), three mantissa bits; exponent 0 is subnormal and
the magnitude code 127 is NaN, so the largest value is 448.
"""
import math

import numpy as np

__all__ = ["FP8_GRID", "code_values", "fp8_quantize", "fp8_values", "fp8_quantize_weight", "fp8_weight_values", "ffn_act"]

#: the values of the magnitude codes 0 .. 126
FP8_GRID = np.array([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7)
                     for e in range(16) for m in range(8)][:127])


def _codes(u):
    """The nearest code of each u (|u| <= 448), the even one on a tie; the sign of u."""
    a = np.abs(u)
    hi = np.clip(np.searchsorted(FP8_GRID, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = FP8_GRID[hi] - a, a - FP8_GRID[lo]
    code = np.where(up < down, hi, np.where(up > down, lo, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(hi == 0, 0, code)
    return (code + 128 * np.signbit(u)).astype(np.uint8)


def _exponent(top):
    """The smallest e in -127 .. with top <= 448 2^e."""
    e = np.full(top.shape, -127)
    for k in range(-127, 122):
        e = np.where(top > np.ldexp(448.0, k), k + 1, e)
    return e


def _bytes(top):
    finite = np.isfinite(top)
    e = _exponent(np.where(finite, top, 0.0))
    return np.where(finite, e + 127, 255).astype(np.uint8), np.ldexp(1.0, e), finite


def fp8_quantize(x):
    """(Q [rows][128 ceil(d / 128)], scale bytes [rows][4 ceil(d / 512)]) of x [rows][d]."""
    x = np.asarray(x, np.float64)
    rows, d = x.shape
    blocks = -(-d // 128)
    p = np.zeros((rows, blocks * 128))
    p[:, :d] = x
    p = p.reshape(rows, blocks, 128)
    byte, scale, finite = _bytes(np.abs(p).max(axis=2))
    Q = np.where(finite[:, :, None], _codes(np.where(finite[:, :, None], p, 0.0) / scale[:, :, None]), 0)
    S = np.full((rows, -(-blocks // 4) * 4), 127, np.uint8)
    S[:, :blocks] = byte
    return Q.reshape(rows, blocks * 128).astype(np.uint8), S


def fp8_quantize_weight(W):
    """(Q [d_out][128 ceil(d_in / 128)], scale bytes [ceil(d_out / 128)][ceil(d_in / 128)])."""
    W = np.asarray(W, np.float64)
    d_out, d_in = W.shape
    rb, cb = -(-d_out // 128), -(-d_in // 128)
    p = np.zeros((rb * 128, cb * 128))
    p[:d_out, :d_in] = W
    p = p.reshape(rb, 128, cb, 128)
    byte, scale, finite = _bytes(np.abs(p).max(axis=(1, 3)))
    ok = finite[:, None, :, None]
    Q = np.where(ok, _codes(np.where(ok, p, 0.0) / scale[:, None, :, None]), 0)
    return Q.reshape(rb * 128, cb * 128)[:d_out].astype(np.uint8), byte


def scale_values(S):
    """float64 scales of bytes (float32 scales as they are)."""
    S = np.asarray(S)
    if S.dtype == np.uint8:
        return np.where(S == 255, np.nan, np.ldexp(1.0, S.astype(np.int64) - 127))
    return S.astype(np.float64)


def code_values(Q):
    Q = np.asarray(Q, np.uint8)
    grid = np.concatenate([FP8_GRID, [np.nan]])
    return grid[Q & 127] * np.where(Q & 128, -1.0, 1.0)


def fp8_values(Q, S, d):
    """float64 values [rows][d] of packed rows."""
    return (code_values(Q) * np.repeat(scale_values(S), 128, axis=1)[:, :Q.shape[1]])[:, :d]


def fp8_weight_values(Q, S, d_in):
    """float64 values [d_out][d_in] of a packed weight."""
    s = np.repeat(np.repeat(scale_values(S), 128, axis=0)[:Q.shape[0]], 128, axis=1)
    return (code_values(Q) * s)[:, :d_in]


def _logistic(z):
    return np.where(z >= 0, 1.0, np.exp(np.minimum(z, 0.0))) / (1 + np.exp(-np.abs(z)))


def ffn_act(z, act):
    """(act(z), act'(z)) in float64, without cancellation in either tail."""
    z = np.asarray(z, np.float64)
    if act == "silu":
        s = _logistic(z)
        return z * s, s + z * s * _logistic(-z)
    if act == "gelu":
        P = 0.5 * np.vectorize(math.erfc)(-z / math.sqrt(2.0))
        return z * P, P + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    # (1 + tanh(u)) / 2 is the logistic function of 2 u
    u = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    s = _logistic(2 * u)
    return z * s, s + 2 * z * s * _logistic(-2 * u) * math.sqrt(2 / math.pi) * (1 + 0.134145 * z * z)
