"""Residual addition + RMS norm in float64, from the definition.

TEST INFRASTRUCTURE ONLY (see the package docstring).
"""

import numpy as np

from .formats import bf16_round


def add_rmsnorm_reference(x, residual, weight, eps, residual_bf16):
    """v = x (+ residual, rounded to bf16 or fp32), n = v * weight / sqrt(mean(v^2) + eps) per row.

    x, residual (or None) and weight are arrays of the exact input values.  Returns (v float64, n float64)."""
    v = np.asarray(x, np.float64)
    if residual is not None:
        # two fp32 (or bf16) values add exactly in float64 unless their exponents lie 29 apart, and then
        # the smaller one cannot move the rounding
        v = (v + np.asarray(residual, np.float64)).astype(np.float32)
        v = (bf16_round(v) if residual_bf16 else v).astype(np.float64)
    n = v * np.asarray(weight, np.float64) / np.sqrt(np.mean(v * v, axis=1, keepdims=True) + eps)
    return v, n
