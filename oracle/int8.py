"""The int8 expert layer's stages in float64 / int64, from the definition.

TEST INFRASTRUCTURE ONLY (see the package docstring).
"""

import numpy as np

from .formats import bf16_round


def int8_product(x, x_scale, w, w_scale):
    """(sum_k x_k w_k) * x_scale[row] * w_scale[channel]; the sums are whole numbers, exact in float64."""
    s = np.asarray(x, np.float64) @ np.asarray(w, np.float64).T
    return s * np.asarray(x_scale, np.float64)[:, None] * np.asarray(w_scale, np.float64)[None]


def swiglu(h):
    I = h.shape[1] // 2
    g, u = h[:, :I], h[:, I:]
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def quantize_rows_int8(v):
    """Codes round(v / s) (ties to even) and s = amax / 127 (1 if zero) per row."""
    v = np.asarray(v, np.float64)
    amax = np.abs(v).max(axis=1)
    s = np.where(amax > 0, amax / 127.0, 1.0)
    return np.rint(v / s[:, None]), s


def moe_reference_int8(x, x_scale, w13, w13_scale, w2, w2_scale, topk_ids, topk_weights):
    """out[t] = sum over valid slots of topk_weight * FFN_expert(x[t]), float64 [T, H]."""
    T = x.shape[0]
    E, H, _ = w2.shape
    out = np.zeros((T, H))
    for e in range(E):
        tok, slot = np.nonzero(topk_ids == e)
        if not tok.size:
            continue
        act = swiglu(int8_product(x[tok], x_scale[tok], w13[e], w13_scale[e]))
        act = bf16_round(act.astype(np.float32)).astype(np.float64)
        q, s = quantize_rows_int8(act)
        y = int8_product(q, s, w2[e], w2_scale[e])
        np.add.at(out, tok, y * np.asarray(topk_weights, np.float64)[tok, slot][:, None])
    return out
