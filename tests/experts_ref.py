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


def blocks(rng, *shape, lo=0.001, hi=0.02):
    """Random Q4_0 blocks uint8 [..., k/32*18] for weights of shape [..., k]."""
    *front, k = shape
    b = rng.integers(0, 256, (*front, k // 32, 18), dtype=np.uint8)
    d = rng.uniform(lo, hi, (*front, k // 32)).astype(np.float16)
    b[..., 0:2] = d[..., None].view(np.uint8)
    return b.reshape(*front, -1)


def matrix(b):
    """float64 weights [..., k], and the scale times (n + 8) of each."""
    b = b.reshape(*b.shape[:-1], -1, 18)
    d = np.ascontiguousarray(b[..., :2]).view(np.float16).astype(np.float64)
    n = np.concatenate([b[..., 2:] & 15, b[..., 2:] >> 4], -1).astype(np.float64)
    flat = (*b.shape[:-2], -1)
    return ((n - 8) * d).reshape(flat), (np.abs(d) * (n + 8)).reshape(flat)


def gelu(z):
    return z / 2 * (1 + np.tanh(np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3)))


def product(x, b, exact, rounded_x):
    """x [rows][k] times the transpose of a matrix of blocks, and the bound of
    the kernels' error.  With S = sum |w x| and T = sum d (n + 8) |x|:
      exact weights (fp32 results): x in two binary16 parts 2^-22, sums of 16
        products in the tensor cores 2^-19 (17 addends cut at 2^-23), K / 32 + 16
        roundings of block sums and parts: 2^-15.9 for K to 8192, 2^-15 S in all,
        and beyond that K 2^-28 S; and of what binary16 cannot reach, 2^-38 of the
        row's largest x for each weight
      bf16 results: an fp32 x in 11 bits, half a step 2^-11; in the streaming
        form sums of subnormal codes that keep 18 bits, 34 addends of T, under
        2^-12 T; in the tile form each weight rounded to binary16, half a step
        2^-12 S and 2^-25 of each x below its normal numbers, and K / 16
        accumulations cut at 2^-23: 2^-14 S for K to 8192, beyond that K 2^-27 S
    """
    w, wide = matrix(b)
    a = np.abs(x)
    s = a @ np.abs(w).T
    reach = 2.0 ** -38 * a.max(-1, keepdims=True) * np.abs(w).sum(-1)
    long = max(1.0, x.shape[-1] / 8192)
    if exact:
        return x @ w.T, s * 2.0 ** -15 * long + reach
    return x @ w.T, (s * (2.0 ** -14 * long + 2.0 ** -12 + (2.0 ** -11 if rounded_x else 0.0)) + a @ wide.T * 2.0 ** -12
                      + a.sum(-1, keepdims=True) * 2.0 ** -25 + reach)


def geglu(x, bg, bu, exact, rounded_x):
    """h and its bound: |gelu'| <= 1.13, the GELU's own evaluation 2^-20 (1 + g^2)."""
    (g, eg), (u, eu) = product(x, bg, exact, rounded_x), product(x, bu, exact, rounded_x)
    h = gelu(g) * u
    return h, (1.13 * np.abs(u) * eg + np.abs(gelu(g)) * eu + 1.13 * eg * eu + 2.0 ** -20 * (1 + g * g) * np.abs(h)
               + (0.0 if exact else 2.0 ** -8 * np.abs(h)) + 1e-37)


def plan_of(ids, experts):
    """expert_start and pairs of ids [tokens][topk], -1 where there is none."""
    flat = ids.reshape(-1)
    there = np.flatnonzero(flat >= 0)
    pairs = np.full(flat.size, -1, dtype=np.int32)
    pairs[:there.size] = there[np.argsort(flat[there], kind="stable")]
    return np.concatenate([[0], np.bincount(flat[there], minlength=experts).cumsum()]).astype(np.int32), pairs


def experts_geglu(x, bg, bu, starts, pairs, topk, exact, rounded_x):
    n = bg.shape[1]
    h, limit = np.zeros((pairs.size, n)), np.zeros((pairs.size, n))
    for e in range(starts.size - 1):
        rows = slice(starts[e], starts[e + 1])
        if rows.start < rows.stop:
            h[rows], limit[rows] = geglu(x[pairs[rows] // topk], bg[e], bu[e], exact, rounded_x)
    return h, limit


def experts_down(h, bd, ids, weights, starts, pairs, exact, rounded_x):
    """y and its bound: the projections' own bounds weighted; the weighted sum
    rounds at most 33 times; z is rounded to bf16 once in the tile form."""
    t, topk = ids.shape
    n = bd.shape[1]
    y, limit = np.zeros((t, n)), np.zeros((t, n))
    w = weights.astype(np.float64).reshape(-1)
    for e in range(starts.size - 1):
        for i in range(starts[e], starts[e + 1]):
            z, ez = product(h[i:i + 1], bd[e], exact, rounded_x)
            p = pairs[i]
            if 0 <= ids.reshape(-1)[p] < starts.size - 1:
                y[p // topk] += w[p] * z[0]
                limit[p // topk] += np.abs(w[p]) * (ez[0] + np.abs(z[0]) * (33 * 2.0 ** -24 + (0.0 if exact else 2.0 ** -8)))
    return y, limit + (0.0 if exact else 2.0 ** -8 * np.abs(y)) + 1e-37
