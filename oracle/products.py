"""The dense and the ragged grouped products and the FP8 block quantiser in float64, from their definitions.

TEST INFRASTRUCTURE ONLY (see the package docstring).
"""

import numpy as np


def block_product(a, a_scale, b, b_scale):
    """sum_k a[m, k] a_scale[m, k // 128] b[n, k] b_scale[n // 128, k // 128]; a and b hold decoded values, scales
    None: plain.  Returns (sums, the sums of the terms' magnitudes)."""
    a, b = np.asarray(a, np.float64), np.asarray(b, np.float64)
    if a_scale is not None:
        a = a * np.asarray(a_scale, np.float64)[:, np.arange(a.shape[1]) // 128]
        b = b * np.asarray(b_scale, np.float64)[np.arange(b.shape[0]) // 128][:, np.arange(b.shape[1]) // 128]
    return a @ b.T, np.abs(a) @ np.abs(b).T


def ragged_product(a, a_scale, b, b_scale, indptr):
    """block_product of rows indptr[e] .. indptr[e + 1] - 1 with b[e]; NaN in rows of no group."""
    rows, N = a.shape[0], b.shape[1]
    y, s = np.full((rows, N), np.nan), np.full((rows, N), np.nan)
    for e in range(b.shape[0]):
        lo, hi = int(indptr[e]), int(indptr[e + 1])
        if hi > lo:
            y[lo:hi], s[lo:hi] = block_product(a[lo:hi], None if a_scale is None else a_scale[lo:hi], b[e],
                                               None if b_scale is None else b_scale[e])
    return y, s


def quant_blocks(v):
    """(v / s, s) per row and 128 columns, s = amax / 448, 1 where that is 0 in fp32; the quotient is not rounded."""
    v = np.asarray(v, np.float64)
    M, N = v.shape
    nb = -(-N // 128)
    s = np.ones((M, nb))
    for k in range(nb):
        amax = np.abs(v[:, 128 * k:128 * (k + 1)]).max(1)
        r = amax / 448.0
        s[:, k] = np.where(r > 2.0 ** -150, r, 1.0)
    return v / s[:, np.arange(N) // 128], s


def silu_mul(x):
    """silu(gate) * up of the halves of x, in float64."""
    g, u = np.split(np.asarray(x, np.float64), 2, axis=1)
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u
