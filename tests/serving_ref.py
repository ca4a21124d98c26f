"""Plain references in 64 bits for the serving operators, on the CPU (numpy),
and the error bounds their tests use.  Nothing here calls the library.

Attention bounds, with A = scale * max_j sum_d |q_d k_jd| over the keys a row
sees and S = sum_j p_j |v_j| (per output):

  fp32 out: a score is formed from binary16 parts of q that together keep 22
  bits (2^-21) and at most 64 fp32 roundings (64 * 2^-24 = 2^-18), so it is
  off by less than A * 2^-17; that shifts each weight by a factor within
  1 +- A * 2^-17, twice (numerator and denominator).  The weights' own
  evaluation, their two parts and the sums over the keys add less than 2^-16.
      |out - ref| <= S * (2 * A * 2^-17 + 2^-16) + 1e-30
      |lse - ref| <= A * 2^-17 + 2^-18 * (1 + |lse|)
  bf16 out: q, k and p enter as one binary16 value each (2^-11 apiece), v as
  one binary16 value, and the output is rounded to bf16 (2^-8 covers it).
      |out - ref| <= S * (4 * A * 2^-11 + 4 * 2^-11) + 2^-8 * |ref| + 1e-30
      |lse - ref| <= 2 * A * 2^-11 + 2^-11 * (1 + |lse|)
"""
import numpy as np


def quantize(x):
    """codes uint8 [..., D/2], scales float16 [..., D/32] of x [..., D] (float32/64)."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(*x.shape[:-1], -1, 32)
    odd = ~np.isfinite(b).all(-1)
    c = np.where(odd[..., None], 0.0, b)
    top, low = c.max(-1), c.min(-1)
    e = np.where(top >= -low, top, low)
    d = np.clip(e / -8, -65504, 65504).astype(np.float32).astype(np.float16)
    f = d.astype(np.float64)[..., None]
    q = np.where(f == 0, 8.0, np.clip(np.rint(c / np.where(f == 0, 1, f)) + 8, 0, 15)).astype(np.uint8)
    q[odd] = 8
    d = np.where(odd, np.float16(np.nan), d).astype(np.float16)
    codes = q[..., :16] | (q[..., 16:] << 4)
    return codes.reshape(*x.shape[:-1], x.shape[-1] // 2), d


def values(codes, scales):
    c = codes.reshape(*codes.shape[:-1], -1, 16)
    n = np.concatenate([c & 15, c >> 4], -1).astype(np.float64) - 8
    return (n * scales.astype(np.float64)[..., None]).reshape(*codes.shape[:-1], -1)


def attention(q, kc, ks, vc, vs, table, q_start, kv_len, scale, causal, window):
    """q float64 [rows][heads][D]; caches as numpy arrays.  Returns out, lse,
    and the A [rows][heads] and S [rows][heads][D] of the bounds."""
    rows, heads, dim = q.shape
    kvh, page = kc.shape[1], kc.shape[2]
    g = heads // kvh
    out = np.zeros((rows, heads, dim))
    lse = np.full((rows, heads), -np.inf)
    big, share = np.zeros((rows, heads)), np.zeros((rows, heads, dim))
    for b, n in enumerate(kv_len):
        n = int(n)
        if n == 0:
            continue
        r0, r1 = int(q_start[b]), int(q_start[b + 1])
        ids = table[b, :-(-n // page)]
        for h in range(kvh):
            k = values(kc[ids, h], ks[ids, h]).reshape(-1, dim)[:n]
            v = values(vc[ids, h], vs[ids, h]).reshape(-1, dim)[:n]
            for r in range(r0, r1):
                pos = n - (r1 - r)
                hi = min(n, pos + 1) if causal else n
                lo = max(0, pos - window + 1) if window else 0
                if hi <= lo:
                    continue
                qq = q[r, h * g:(h + 1) * g]
                s = qq @ k[lo:hi].T * scale
                m = s.max(-1, keepdims=True)
                w = np.exp(s - m)
                l = w.sum(-1, keepdims=True)
                p = w / l
                out[r, h * g:(h + 1) * g] = p @ v[lo:hi]
                lse[r, h * g:(h + 1) * g] = (m + np.log(l))[:, 0]
                big[r, h * g:(h + 1) * g] = (np.abs(qq) @ np.abs(k[lo:hi]).T).max(-1) * abs(scale)
                share[r, h * g:(h + 1) * g] = p @ np.abs(v[lo:hi])
    return out, lse, big, share


def attention_limits(out, lse, big, share, bf16):
    a = big[..., None]
    finite = np.where(np.isfinite(lse), np.abs(lse), 0.0)
    if bf16:
        return (share * (4 * a + 4) * 2.0 ** -11 + 2.0 ** -8 * np.abs(out) + 1e-30,
                2 * big * 2.0 ** -11 + 2.0 ** -11 * (1 + finite))
    return share * (2 * a * 2.0 ** -17 + 2.0 ** -16) + 1e-30, big * 2.0 ** -17 + 2.0 ** -18 * (1 + finite)


def plan(cached, added, free, table, page, capacity):
    table = table.copy()
    width, at, slots, pos, q_start = table.shape[1], 0, [], [], [0]
    for b, (c, a) in enumerate(zip(cached, added)):
        first, last = -(-c // page), -(-(c + a) // page)
        for i in range(first, last):
            if i < width:
                table[b, i] = free[at] if at < len(free) else -1
            at += 1
        for p in range(c, c + a):
            held = table[b, p // page] if p // page < width else -1
            slots.append(held * page + p % page if held >= 0 else -1)
            pos.append(p)
        q_start.append(min(len(slots), capacity))
    pad = [-1] * max(0, capacity - len(slots))
    return (table, np.array(q_start), np.array(cached) + np.array(added),
            np.array((slots + pad)[:capacity]), np.array((pos + pad)[:capacity]), np.array([at]))


def logits(x, history, prompt, rep, freq, pres, bias, allowed):
    """history: list of id arrays; bias: list of (id, value) lists; allowed: bool [rows][vocab] or None."""
    y = x.astype(np.float64)
    rows, vocab = y.shape
    for i in range(rows):
        ids = history[i]
        keep = (ids >= 0) & (ids < vocab)
        seen, made = np.zeros(vocab), np.zeros(vocab)
        np.add.at(seen, ids[keep], 1)
        late = keep & (np.arange(len(ids)) >= prompt[i])
        np.add.at(made, ids[late], 1)
        y[i] = np.where(seen > 0, np.where(y[i] > 0, y[i] / rep[i], y[i] * rep[i]), y[i])
        y[i] -= made * freq[i] + (made > 0) * pres[i]
        for t, v in bias[i]:
            if 0 <= t < vocab:
                y[i, t] += v
        if allowed is not None:
            y[i, ~allowed[i]] = -np.inf
    return y
