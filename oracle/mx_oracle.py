"""fp64 CPU oracle for the MXFP4 rows.

TEST INFRASTRUCTURE ONLY, like gq_oracle: NumPy, float64, the plain definitions of the OCP
Microscaling format's e2m1 elements with e8m0 scales over blocks of 32.

Layout of a row of d values: codes two to a byte (even element low), zero codes up to a
multiple of 128 values; one scale byte a block, 127 past the last one.
"""
import numpy as np

__all__ = ["mx_quantize", "mx_values", "MX_GRID"]

MX_GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def mx_quantize(x):
    """(Q, S) of x [rows][d]: per block the scale 2^e, e = clamp(floor(log2 max|x|) - 2, -127,
    125), and per value the nearest of the grid in units of it (the even index on a tie)."""
    x = np.asarray(x, np.float64)
    rows, d = x.shape
    groups = -(-d // 128)
    Q = np.zeros((rows, groups * 128), np.uint8)
    S = np.full((rows, groups * 4), 127, np.uint8)
    for b in range(-(-d // 32)):
        v = x[:, 32 * b:32 * b + 32]
        top = np.abs(v).max(axis=1)
        finite = np.isfinite(top)
        safe = np.where(finite & (top > 0), top, 2.0 ** -200)
        e = np.clip(np.frexp(safe)[1] - 1 - 2, -127, 125)     # frexp: top = m 2^k, m in [1/2, 1)
        u = np.where(finite[:, None], v, 0.0) / np.ldexp(1.0, e)[:, None]
        far = np.abs(np.abs(u)[:, :, None] - MX_GRID)
        least = far.min(axis=2, keepdims=True)
        code = np.zeros(u.shape, np.int64)
        done = np.zeros(u.shape, bool)
        for k in (0, 2, 4, 6, 1, 3, 5, 7):                    # the even index keeps a tie
            hit = (far[:, :, k] == least[:, :, 0]) & ~done
            code[hit] = k
            done |= hit
        code += 8 * (np.signbit(u) & finite[:, None])
        Q[:, 32 * b:32 * b + 32][:, :v.shape[1]] = code
        S[:, b] = np.where(finite, e + 127, 255)
    return Q[:, 0::2] | (Q[:, 1::2] << 4), S


def mx_values(Q, S, d):
    """float64 values [rows][d] of packed rows (NaN where the scale byte is 255)."""
    Q, S = np.asarray(Q, np.uint8), np.asarray(S, np.uint8)
    code = np.stack([Q & 15, Q >> 4], axis=2).reshape(Q.shape[0], -1)[:, :d]
    v = MX_GRID[code & 7] * np.where(code & 8, -1.0, 1.0)
    scale = np.where(S == 255, np.nan, np.ldexp(1.0, S.astype(np.int64) - 127))
    return v * np.repeat(scale, 32, axis=1)[:, :d]
