"""Plain references in 64 bits for the operators of a mixture-of-experts layer,
on the CPU (numpy), and the error bounds their tests use.  Nothing here calls
the library.
"""
import numpy as np


def turn(x, table, positions, rot, interleaved):
    """x [n][heads][dim] rotated by rows of table, each product and sum rounded
    once to float32 (numpy does not contract).  Rows of position -1 as they are."""
    x = np.asarray(x, dtype=np.float32)
    out = x.copy()
    first = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    second = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    for i, p in enumerate(positions):
        if p < 0:
            continue
        c, s = table[p, :rot // 2], table[p, rot // 2:]
        a, b = x[i][:, first], x[i][:, second]
        out[i][:, first] = (a * c).astype(np.float32) - (b * s).astype(np.float32)
        out[i][:, second] = (a * s).astype(np.float32) + (b * c).astype(np.float32)
    return out


def _order(v):
    """Indices by falling value, equals by index, NaN behind -inf."""
    nan = np.isnan(v)
    return np.lexsort((np.arange(v.size), -np.where(nan, -np.inf, v), nan))


def route(logits, bias, topk, score, groups=1, group_topk=1, group_best=1, renormalize=True, scale=1.0, count=None):
    """ids, weights, expert_start, pairs."""
    x = np.asarray(logits, dtype=np.float64)
    tokens, experts = x.shape
    real = tokens if count is None else min(max(count, 0), tokens)
    ids = np.full((tokens, topk), -1, dtype=np.int64)
    weights = np.zeros((tokens, topk))
    size = experts // groups
    with np.errstate(all="ignore"):
        for t in range(real):
            if score == "sigmoid":
                s = 1 / (1 + np.exp(-x[t]))
            else:
                top = np.nanmax(np.append(x[t], -np.inf))
                w = np.exp(x[t] - (top if top > -np.inf else 0.0))
                s = w / w.sum() if w.sum() != 0 else np.zeros(experts)
            c = s + np.asarray(bias, dtype=np.float64) if bias is not None else s
            rank = c if bias is not None else x[t]
            if groups > 1:
                g = np.array([np.sort(v[~np.isnan(v)])[::-1][:group_best].sum() if (~np.isnan(v)).any() else -np.inf
                              for v in (rank if group_best == 1 else c).reshape(groups, size)])
                kept = _order(g)[:group_topk]
                within = np.flatnonzero(np.isin(np.arange(experts) // size, kept))
            else:
                within = np.arange(experts)
            ids[t] = within[_order(rank[within])[:topk]]
            w = s[ids[t]]
            if renormalize:
                w = w / w.sum() if w.sum() != 0 else w * 0
            weights[t] = w * scale
    flat = ids.reshape(-1)
    there = np.flatnonzero(flat >= 0)
    pairs = np.full(tokens * topk, -1)
    pairs[:there.size] = there[np.argsort(flat[there], kind="stable")]
    starts = np.concatenate([[0], np.bincount(flat[there], minlength=experts).cumsum()])
    return ids, weights, starts, pairs


# Weights: a score is off by less than (8 + 40 + |l - top|) 2^-24 of itself
# (exponential, its argument, sum of at most 1024 terms in 37 levels, division),
# |l - top| at most 40 in the tests; their quotient by a sum by twice that and
# 10 roundings.  2 (8 + 40 + 40) + 10 < 2^8 units of 2^-24.
WEIGHT = 2.0 ** -16
