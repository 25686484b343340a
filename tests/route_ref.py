"""Routing from its definition (include/dqmoe.h, dq_moe_routing) in plain Python and 64 bits, a token at a time."""
import numpy as np


def route(logits, top_k, scores="softmax", bias=None, n_groups=1, top_groups=1, group_score="max", renormalize=True,
          scale=1.0):
    """logits [T][E] (any float type) -> (idx [T][top_k], gate [T][top_k] as float64)."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    idx, gate = np.zeros((T, top_k), dtype=np.int32), np.zeros((T, top_k))
    per = E // n_groups
    for t in range(T):
        l = np.where(np.isnan(logits[t]), -np.inf, np.minimum(logits[t], np.finfo(np.float32).max))
        live = l > -np.inf
        with np.errstate(over="ignore", under="ignore"):
            if scores == "sigmoid":
                s = np.where(live, 1.0 / (1.0 + np.exp(-np.where(live, l, 0.0))), 0.0)
            else:
                w = np.where(live, np.exp(np.where(live, l, 0.0) - (l[live].max() if live.any() else 0.0)), 0.0)
                s = w / w.sum() if live.any() else w
        v = s + (0.0 if bias is None else np.asarray(bias, dtype=np.float64))
        if bias is None:
            v = l.copy()                         # scores rise with the logits, which differ where scores may not
        v = np.where(live, v, -np.inf)
        for_sum = np.where(live, s if bias is None else v, -np.inf)
        group = []
        for g in range(n_groups):
            if group_score == "max":
                group.append(v[g * per:(g + 1) * per].max())
            else:
                two = np.sort(for_sum[g * per:(g + 1) * per])[::-1][:2]
                group.append(two[two > -np.inf].sum() if (two > -np.inf).any() else -np.inf)
        kept = sorted(range(n_groups), key=lambda g: (-group[g], g))[:top_groups]
        ok = np.zeros(E, dtype=bool)
        for g in kept:
            ok[g * per:(g + 1) * per] = True
        v = np.where(ok, v, -np.inf)
        pick = sorted(range(E), key=lambda e: (-v[e], e))[:top_k]
        idx[t] = pick
        x = np.where(v[pick] > -np.inf, s[pick], 0.0)
        gate[t] = scale * (x / (x.sum() + 1e-20) if renormalize else x)
    return idx, gate
