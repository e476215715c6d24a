"""The router's choice of experts in float64, token by token, from the definition.

TEST INFRASTRUCTURE ONLY (see the package docstring).
"""

import numpy as np


def router_reference(logits, K, score, bias=None, n_group=1, topk_group=1, group_top=1, renormalize=True, scale=1.0):
    """logits [T, E] (exact input values), score "softmax" or "sigmoid".
    Returns (ids int32 [T, K], weights float64 [T, K]); -1 and 0 in slots no expert is left for."""
    x = np.asarray(logits, np.float64)
    T, E = x.shape
    ids = np.full((T, K), -1, np.int32)
    weights = np.zeros((T, K))
    for t in range(T):
        able = ~(np.isnan(x[t]) | (x[t] == -np.inf))
        sc = np.zeros(E)
        if able.any():
            if score == "softmax":
                m = x[t][able].max()
                with np.errstate(invalid="ignore"):
                    p = np.where(x[t][able] == m, 1.0, np.exp(x[t][able] - m))
                sc[able] = p / p.sum()
            else:
                with np.errstate(over="ignore"):
                    sc[able] = 1.0 / (1.0 + np.exp(-x[t][able]))
        choice = sc + np.asarray(bias, np.float64) if bias is not None else x[t].copy()
        able &= ~(np.isnan(choice) | (choice == -np.inf))
        choice[~able] = -np.inf
        if n_group > 1:
            inside = choice if bias is not None or group_top == 1 else np.where(able, sc, -np.inf)
            best = -np.sort(-inside.reshape(n_group, -1), axis=1)[:, :group_top]
            # a group of fewer experts than group_top counts as -inf
            best = np.where((best == -np.inf).any(axis=1), -np.inf, np.where(best == -np.inf, 0, best).sum(axis=1))
            kept = np.lexsort((np.arange(n_group), -best))[:topk_group]
            out = ~np.isin(np.arange(E) // (E // n_group), kept)
            able &= ~out
        order = [e for e in np.lexsort((np.arange(E), -choice)) if able[e]][:K]
        ids[t, :len(order)] = order
        w = sc[order]
        if renormalize:
            w = w / w.sum() if w.sum() > 0 else np.zeros_like(w)
        weights[t, :len(order)] = w * scale
    return ids, weights
