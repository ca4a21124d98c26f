"""The serving operators around the quantized products, as measured cases.

Four operators of a decode or prefill step over a paged cache of keys and
values held in Q4_0 (4-bit codes and one binary16 scale per 32 values):

  plan    page tables and slot maps from the requests' lengths
  append  new keys and values quantized into the cache and read back
  attn    attention over the cache, for single tokens and for prompts
  logits  penalties, biases and grammar masks on the LM head's logits

Each has a plain form in elementary torch operations (fp32, one rounding at
the end) and the library's own call; `own` chooses between them.
"""
import math
import random

import torch

own = False

DEV = "cuda"


def _qmm():
    from block_quantized_matmul_gguf_gb300 import qmm
    return qmm


# ---- cases --------------------------------------------------------------------

def listed():
    return [
        # sixteen requests that each decode one token: the call that a serving
        # loop makes before every step, pure latency
        {"name": "plan-decode-16", "op": "plan", "batch": 16, "cached": 4000, "added": 1, "page": 64},
        # continuous batching with chunked prompts: a thousand requests, some
        # with one token and some with several hundred
        {"name": "plan-mixed-1001", "op": "plan", "batch": 1001, "cached": 3000, "added": 511, "page": 16},
        # the keys and values of one decode step of sixteen requests: 2 heads
        # of 256 (the decode layer's 512-row k and v projections), fp32
        {"name": "append-decode-16", "op": "append", "tokens": 16, "kv_heads": 2, "dim": 256, "page": 64, "dtype": "f32"},
        # a long prompt's keys and values, an odd number of tokens
        {"name": "append-prompt-8191", "op": "append", "tokens": 8191, "kv_heads": 2, "dim": 256, "page": 64, "dtype": "f32"},
        # one request with a short context: latency
        {"name": "attn-one-301", "op": "attn", "batch": 1, "ctx": 301, "new": 1, "heads": 8, "kv_heads": 2, "dim": 256, "page": 64, "window": 0, "dtype": "f32"},
        # a batch of sixteen requests of uneven lengths, one token each: the
        # largest batch of the fp32 GEMV
        {"name": "attn-batch-16", "op": "attn", "batch": 16, "ctx": 4097, "new": 1, "heads": 8, "kv_heads": 2, "dim": 256, "page": 64, "window": 0, "dtype": "f32"},
        # one long context: the split of one request over the whole GPU
        {"name": "attn-long-131071", "op": "attn", "batch": 1, "ctx": 131071, "new": 1, "heads": 8, "kv_heads": 2, "dim": 256, "page": 16, "window": 0, "dtype": "f32"},
        # many requests at once in bf16: the bandwidth of the 4-bit cache
        {"name": "attn-serve-128", "op": "attn", "batch": 128, "ctx": 8192, "new": 1, "heads": 16, "kv_heads": 4, "dim": 128, "page": 64, "window": 0, "dtype": "bf16"},
        # a 2048-token chunk of a prompt behind 6000 cached tokens
        {"name": "attn-prompt-2048", "op": "attn", "batch": 1, "ctx": 8048, "new": 2048, "heads": 8, "kv_heads": 2, "dim": 256, "page": 64, "window": 0, "dtype": "bf16"},
        # prompts and single tokens in one call, with a sliding window
        {"name": "attn-mixed-window", "op": "attn", "batch": 7, "ctx": 4500, "new": 700, "heads": 16, "kv_heads": 4, "dim": 128, "page": 32, "window": 1024, "dtype": "bf16"},
        # the 262144 logits of one request, with a short history
        {"name": "logits-one", "op": "logits", "rows": 1, "vocab": 262144, "history": 500, "bias": 10, "mask": True},
        # a batch of requests with long histories and an odd vocabulary
        {"name": "logits-batch-64", "op": "logits", "rows": 64, "vocab": 262143, "history": 8000, "bias": 100, "mask": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "attn", "attn", "prompt", "logits"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        return {"op": op, "batch": _log(rng, 1, 2000), "cached": _log(rng, 1, 8000),
                "added": rng.choice([1, _log(rng, 2, 600)]), "page": page}
    if op == "append":
        return {"op": op, "tokens": _log(rng, 1, 8191), "kv_heads": rng.choice([1, 2, 4]),
                "dim": rng.choice([64, 128, 256]), "page": page, "dtype": rng.choice(["f32", "bf16"])}
    if op == "logits":
        return {"op": op, "rows": _log(rng, 1, 64), "vocab": _log(rng, 30000, 262144),
                "history": _log(rng, 1, 8000), "bias": _log(rng, 1, 300), "mask": rng.choice([True, False])}
    kv, group, dim = rng.choice([1, 2, 4]), rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256])
    dtype = rng.choice(["f32", "bf16"])
    if op == "attn":  # single tokens, or the few that speculation verifies
        batch, ctx = _log(rng, 1, 128), _log(rng, 16, 131071)
        ctx = max(16, min(ctx, (1 << 29) // (batch * kv * dim)))
        return {"op": "attn", "batch": batch, "ctx": ctx, "new": rng.choice([1, 1, 2, 4]), "heads": kv * group,
                "kv_heads": kv, "dim": dim, "page": page, "window": rng.choice([0, 0, 512]), "dtype": dtype}
    batch, new = rng.choice([1, 1, 2, 5]), _log(rng, 17, 2048)  # prompts
    ctx = new + _log(rng, 1, 6000)
    while batch * new * ctx * kv * group * dim > 2048 * 8048 * 8 * 256:
        new = max(1, new // 2)
        ctx = max(new, ctx // 2)
    return {"op": "attn", "batch": batch, "ctx": ctx, "new": new, "heads": kv * group, "kv_heads": kv,
            "dim": dim, "page": page, "window": rng.choice([0, 0, 1024]), "dtype": "bf16"}


def _lengths(case):
    """(cached, added) tokens of each request, from the case alone."""
    r = random.Random(str(sorted((k, str(v)) for k, v in case.items() if k != "name")))
    n = case["batch"]
    if case["op"] == "plan":
        cached = [r.randint(0, case["cached"]) for _ in range(n)]
        added = [1 if r.random() < 0.5 else r.randint(1, case["added"]) for _ in range(n)]
        return cached, added
    top, new = case["ctx"], case["new"]
    added = [new if i == 0 or new <= 4 or r.random() < 0.6 else r.randint(1, new) for i in range(n)]
    total = [top if i == 0 else max(added[i], r.randint(max(1, top // 8), top)) for i in range(n)]
    return [t - a for t, a in zip(total, added)], added


def _pages(tokens, page):
    return -(-tokens // page)


# ---- inputs --------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _quantize(x):
    """Q4_0 codes [..., D/2] and scales [..., D/32] of x [..., D] (fp32)."""
    b = x.unflatten(-1, (-1, 32))
    top, low = b.amax(-1), b.amin(-1)
    extreme = torch.where(top >= -low, top, low)
    d = (extreme / -8).clamp(-65504.0, 65504.0).half()
    f = d.float()[..., None]
    q = torch.where(f == 0, torch.full_like(b, 8.0), (torch.round(b / f) + 8).clamp(0, 15)).to(torch.uint8)
    return (q[..., :16] | (q[..., 16:] << 4)).flatten(-2), d


def _values(codes, scales):
    """The fp32 values [..., D] that codes and scales stand for."""
    c = codes.unflatten(-1, (-1, 16))
    n = torch.cat([c & 15, c >> 4], -1).float() - 8
    return (n * scales.float()[..., None]).flatten(-2)


def _random_cache(g, pages, case):
    """One of the two halves of a filled cache, as a program has it in hand."""
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    x = torch.randn(shape, generator=g, device=DEV)
    x *= 1 + 3 * (torch.rand(case["kv_heads"], 1, case["dim"], generator=g, device=DEV) < 0.03)  # strong channels
    return _quantize(x)


def prepare(case, seed):
    g = _gen(seed)
    s = {"op": case["op"], "case": case}
    if case["op"] == "plan":
        cached, added = _lengths(case)
        page = case["page"]
        width = max(_pages(c + a, page) for c, a in zip(cached, added)) + 3
        had = sum(_pages(c, page) for c in cached)
        take = sum(_pages(c + a, page) - _pages(c, page) for c, a in zip(cached, added))
        ids = torch.randperm(had + take + 50, generator=g, device=DEV).int()
        # the pages that the requests hold, then the free list
        grid = torch.arange(width, device=DEV)[None]
        held = _i32([_pages(c, page) for c in cached])
        first = held.cumsum(0) - held
        at = (first[:, None] + grid).clamp(max=max(had - 1, 0))
        table = torch.where(grid < held[:, None], ids[at], -1).int().contiguous()
        cap = sum(added) + 7  # a fixed capacity, as for a captured graph
        s.update(cached=_i32(cached), added=_i32(added), free=ids[had:].contiguous(), table=table, page=page,
                 q_start=torch.empty(case["batch"] + 1, dtype=torch.int32, device=DEV),
                 kv_len=torch.empty(case["batch"], dtype=torch.int32, device=DEV),
                 slots=torch.empty(cap, dtype=torch.int64, device=DEV),
                 positions=torch.empty(cap, dtype=torch.int32, device=DEV),
                 taken=torch.empty(1, dtype=torch.int32, device=DEV))
    elif case["op"] == "append":
        n, kv, dim, page = case["tokens"], case["kv_heads"], case["dim"], case["page"]
        pages = _pages(n, page) + 5
        order = torch.randperm(pages, generator=g, device=DEV)
        token = torch.arange(n, device=DEV)
        # k and v lie side by side in one projection's output
        both = torch.randn(n, 2, kv, dim, generator=g, device=DEV).to(_dtype(case))
        s.update(k=both[:, 0], v=both[:, 1], slots=order[token // page] * page + token % page,
                 codes=[torch.zeros(pages, kv, page, dim // 2, dtype=torch.uint8, device=DEV) for _ in range(2)],
                 scales=[torch.zeros(pages, kv, page, dim // 32, dtype=torch.float16, device=DEV) for _ in range(2)],
                 out=[torch.empty(n, kv, dim, device=DEV) for _ in range(2)])
    elif case["op"] == "attn":
        cached, added = _lengths(case)
        page = case["page"]
        need = [_pages(c + a, page) for c, a in zip(cached, added)]
        pages = sum(need) + 3
        ids = torch.randperm(pages, generator=g, device=DEV).int()
        grid, n = torch.arange(max(need), device=DEV)[None], _i32(need)
        at = (n.cumsum(0) - n)[:, None] + grid
        table = torch.where(grid < n[:, None], ids[at.clamp(max=pages - 1)], -1).int().contiguous()
        (kc, ks), (vc, vs) = _random_cache(g, pages, case), _random_cache(g, pages, case)
        total, heads, dim = sum(added), case["heads"], case["dim"]
        q = torch.randn(total, heads, dim, generator=g, device=DEV).to(_dtype(case))
        ends = [0]
        for a in added:
            ends.append(ends[-1] + a)
        s.update(codes=[kc, vc], scales=[ks, vs], table=table, q=q, q_start=_i32(ends),
                 kv_len=_i32([c + a for c, a in zip(cached, added)]), max_q=max(added), scale=dim ** -0.5,
                 window=case["window"], out=torch.empty_like(q),
                 lse=torch.empty(total, heads, dtype=torch.float32, device=DEV))
    else:
        m, vocab, top = case["rows"], case["vocab"], case["history"]
        r = random.Random(str(sorted((k, str(v)) for k, v in case.items() if k != "name")))
        lens = [top if i == 0 else r.randint(0, top) for i in range(m)]
        ends = [0]
        for a in lens:
            ends.append(ends[-1] + a)
        # tokens repeat as text does: few ids hold most of a history
        u = torch.rand(ends[-1], generator=g, device=DEV)
        history = (u.pow(4) * vocab).int().clamp(max=vocab - 1)
        nb = case["bias"]
        ids = torch.stack([torch.randperm(vocab, generator=g, device=DEV)[:nb] for _ in range(m)]).int()
        words = torch.randint(0, 1 << 32, (m, _pages(vocab, 32)), generator=g, device=DEV, dtype=torch.int64)
        words = torch.where(words >= 1 << 31, words - (1 << 32), words).int()
        s.update(logits=torch.randn(m, vocab, generator=g, device=DEV) * 3, history=history, hist_start=_i32(ends),
                 prompt_len=_i32([n // 2 for n in lens]),
                 repetition=1 + torch.rand(m, generator=g, device=DEV) * 0.5,
                 frequency=torch.rand(m, generator=g, device=DEV) * 0.3,
                 presence=torch.rand(m, generator=g, device=DEV) * 0.5,
                 bias_ids=ids.flatten().contiguous(), bias_values=torch.randn(m * nb, generator=g, device=DEV) * 2,
                 bias_start=_i32([i * nb for i in range(m + 1)]), allowed=words if case["mask"] else None,
                 out=torch.empty(m, vocab, device=DEV))
    if own:  # the handle and the workspace that a program makes once
        if case["op"] in ("append", "attn"):
            s["cache"] = _qmm().KvCacheQ4_0(s["codes"][0], s["scales"][0], s["codes"][1], s["scales"][1])
        if case["op"] == "attn":
            s["workspace"] = _qmm().attn_workspace(s["cache"], case["heads"])
    return s


# ---- one pass --------------------------------------------------------------------

def run(state):
    return (_own if own else _plain)[state["op"]](state)


def _own_plan(s):
    _qmm().qmm_kv_plan(s["cached"], s["added"], s["free"], s["table"], s["page"], s["q_start"], s["kv_len"],
                       s["slots"], s["positions"], s["taken"])
    return [s["table"], s["q_start"], s["kv_len"], s["slots"], s["positions"], s["taken"]]


def _own_append(s):
    q = _qmm()
    q.qmm_kv_append_q4_0(s["cache"], s["k"], s["v"], s["slots"])
    q.qmm_kv_read_q4_0(s["cache"], s["slots"], s["out"][0], s["out"][1])
    return [s["out"][0], s["out"][1]]


def _own_attn(s):
    _qmm().qmm_attn_q4_0(s["cache"], s["q"], s["out"], s["table"], s["q_start"], s["kv_len"], s["max_q"], s["scale"],
                         causal=True, window=s["window"], lse=s["lse"], workspace=s["workspace"])
    return [s["out"], s["lse"]]


def _own_logits(s):
    _qmm().qmm_logits_adjust(s["logits"], s["out"], history=s["history"], hist_start=s["hist_start"],
                             prompt_len=s["prompt_len"], repetition=s["repetition"], frequency=s["frequency"],
                             presence=s["presence"], bias_ids=s["bias_ids"], bias_values=s["bias_values"],
                             bias_start=s["bias_start"], allowed=s["allowed"])
    return [s["out"]]


_own = {"plan": _own_plan, "append": _own_append, "attn": _own_attn, "logits": _own_logits}


def _plain_plan(s):
    page, cached, added, table = s["page"], s["cached"], s["added"], s["table"]
    width, cap, nfree = table.shape[1], s["slots"].numel(), s["free"].numel()
    zero = torch.zeros(1, dtype=torch.int64, device=DEV)
    q_start = torch.cat([zero, added.cumsum(0)]).int()
    kv_len = cached + added
    before, after = (cached + page - 1) // page, (kv_len + page - 1) // page
    need = after - before
    first = need.cumsum(0) - need
    grid = torch.arange(width, device=DEV)[None]
    new = (grid >= before[:, None]) & (grid < after[:, None])
    at = first[:, None] + grid - before[:, None]
    ids = torch.where(at < nfree, s["free"][at.clamp(0, nfree - 1)], -1)
    table = torch.where(new, ids, table).int()
    t = torch.arange(cap, device=DEV)
    real = t < q_start[-1]
    req = torch.searchsorted(q_start[1:].contiguous(), t.int(), right=True).clamp(max=added.numel() - 1)
    pos = cached[req] + t - q_start[req]
    held = table[req, (pos // page).clamp(0, width - 1)].long()
    slots = torch.where(real & (held >= 0), held * page + pos % page, -1)
    return [table, q_start, kv_len, slots, torch.where(real, pos, -1).int(), need.sum().int().reshape(1)]


def _plain_append(s):
    out = []
    for half, x in enumerate((s["k"], s["v"])):
        codes, scales = _quantize(x.float())
        page = s["case"]["page"]
        at, off = s["slots"] // page, s["slots"] % page
        s["codes"][half][at, :, off] = codes
        s["scales"][half][at, :, off] = scales
        out.append(_values(s["codes"][half][at, :, off], s["scales"][half][at, :, off]))
    return out


def _plain_attn(s):
    b, heads, dim = s["kv_len"].numel(), s["q"].shape[1], s["q"].shape[2]
    kv = s["codes"][0].shape[1]
    pages = s["table"].clamp(min=0).long()
    k, v = (_values(c[pages], d[pages]).transpose(1, 2).flatten(2, 3) for c, d in zip(s["codes"], s["scales"]))
    kv_len, q_start = s["kv_len"].long(), s["q_start"].long()
    n, mq = k.shape[2], s["max_q"]
    i = torch.arange(mq, device=DEV)
    rows = (q_start[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][rows].float().unflatten(2, (kv, heads // kv)).permute(0, 2, 3, 1, 4)  # b, kv, group, i, dim
    pos = (kv_len - (q_start[1:] - q_start[:-1]))[:, None] + i
    j = torch.arange(n, device=DEV)
    seen = (j <= pos[:, :, None]) & (j < kv_len[:, None, None])
    if s["window"]:
        seen &= j > pos[:, :, None] - s["window"]
    v = torch.where((j < kv_len[:, None])[:, None, :, None], v, 0.0)
    w = (q.flatten(2, 3) @ k.transpose(2, 3) * s["scale"]).unflatten(2, (heads // kv, mq))
    w = w.masked_fill(~seen[:, None, None], -math.inf)
    top = w.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    w = torch.exp(w - top)
    total = w.sum(-1)
    out = (w.flatten(2, 3) @ v).unflatten(2, (heads // kv, mq)) / torch.where(total == 0, 1.0, total)[..., None]
    lse = top[..., 0] + torch.log(total)
    t = torch.arange(s["q"].shape[0], device=DEV)
    req = torch.searchsorted(s["q_start"][1:].contiguous(), t.int(), right=True)
    at = t - q_start[req]
    out = out.flatten(1, 2)[req, :, at]
    return [out.to(s["q"].dtype), lse.flatten(1, 2)[req, :, at].contiguous()]


def _plain_logits(s):
    x = s["logits"]
    m, vocab = x.shape
    t = torch.arange(s["history"].numel(), device=DEV)
    row = torch.searchsorted(s["hist_start"][1:].contiguous(), t.int(), right=True)
    made = (t - s["hist_start"][row] >= s["prompt_len"][row]).float()
    at = row * vocab + s["history"]
    seen = torch.zeros(m * vocab, device=DEV).index_fill_(0, at, 1.0).view(m, vocab)
    count = torch.zeros(m * vocab, device=DEV).index_add_(0, at, made).view(m, vocab)
    r = s["repetition"][:, None]
    y = torch.where(seen > 0, torch.where(x > 0, x / r, x * r), x)
    y = y - (count * s["frequency"][:, None] + (count > 0) * s["presence"][:, None])
    b = torch.arange(s["bias_ids"].numel(), device=DEV)
    brow = torch.searchsorted(s["bias_start"][1:].contiguous(), b.int(), right=True)
    y = y.reshape(-1).index_add(0, brow * vocab + s["bias_ids"], s["bias_values"]).view(m, vocab)
    if s["allowed"] is not None:
        bit = torch.arange(vocab, device=DEV)
        y = y.masked_fill(((s["allowed"][:, bit // 32] >> (bit % 32).int()) & 1) == 0, -math.inf)
    return [y]


_plain = {"plan": _plain_plan, "append": _plain_append, "attn": _plain_attn, "logits": _plain_logits}


# ---- what a pass cannot do without --------------------------------------------------

def work(case):
    if case["op"] == "plan":
        cached, added = _lengths(case)
        n, t = case["batch"], sum(added)
        take = sum(_pages(c + a, case["page"]) - _pages(c, case["page"]) for c, a in zip(cached, added))
        # lengths in; starts and lengths out; 12 bytes a token; each new page read and written
        return {"bytes": 8 * n + 8 * n + 12 * t + 8 * take, "flops": 0}
    if case["op"] == "append":
        n = case["tokens"] * case["kv_heads"] * case["dim"] * 2
        # inputs, the cache written and read once (18 bytes per 32 values), the values out, the slots twice
        return {"bytes": n * (4 if case["dtype"] == "f32" else 2) + 2 * n * 18 // 32 + 4 * n + 16 * case["tokens"],
                "flops": 4 * n}
    if case["op"] == "attn":
        cached, added = _lengths(case)
        size, w = (4 if case["dtype"] == "f32" else 2), case["window"]
        keys = pairs = 0
        for c, a in zip(cached, added):
            keys += c + a if not w else c + a - max(0, c - w + 1)
            for_one = [min(c + i + 1, w) if w else c + i + 1 for i in range(a)]
            pairs += sum(for_one)
        rows = sum(added) * case["heads"]
        return {"bytes": keys * case["kv_heads"] * case["dim"] * 2 * 18 // 32 + 2 * rows * case["dim"] * size + 4 * rows,
                "flops": 4 * pairs * case["heads"] * case["dim"]}
    m, vocab = case["rows"], case["vocab"]
    n = m * vocab
    history = case["history"] * (1 + (m - 1) / 2)  # the rows after the first have half of it on average
    return {"bytes": 8 * n + (n // 8 if case["mask"] else 0) + 4 * history + 8 * m * case["bias"], "flops": 5 * n}


# ---- the definition, in 64 bits ------------------------------------------------------

def _exact_values(codes, scales):
    """Byte i of a block holds value i in its low and value i + 16 in its high four bits."""
    out = torch.empty(*codes.shape[:-1], codes.shape[-1] // 16, 32, dtype=torch.float64, device=DEV)
    c = codes.unflatten(-1, (-1, 16))
    out[..., :16] = (c % 16).double()
    out[..., 16:] = torch.div(c, 16, rounding_mode="floor").double()
    return ((out - 8) * scales.double()[..., None]).flatten(-2)


def _exact_append(s):
    got = []
    for x in (s["k"], s["v"]):
        b = x.double().unflatten(-1, (-1, 32))
        size, at = b.abs().max(-1)
        extreme = b.gather(-1, at[..., None])[..., 0]
        extreme = torch.where(b.amax(-1) == size, size, extreme)  # of +a and -a, the positive one
        d = (extreme / -8).clamp(-65504, 65504).half().double()[..., None]
        n = torch.where(d == 0, 0.0, torch.round(b / torch.where(d == 0, 1.0, d)).clamp(-8, 7))
        got.append((n * d).flatten(-2))
    return got


def _exact_attn(s):
    case = s["case"]
    group, page = case["heads"] // case["kv_heads"], case["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    start, lens = s["q_start"].tolist(), s["kv_len"].tolist()
    for r, n in enumerate(lens):
        lo, hi = start[r], start[r + 1]
        ids = s["table"][r, :_pages(n, page)].long()
        for h in range(case["kv_heads"]):
            k, v = (_exact_values(c[ids, h], d[ids, h]).flatten(0, 1)[:n] for c, d in zip(s["codes"], s["scales"]))
            q = s["q"][lo:hi, h * group:(h + 1) * group].double()
            score = torch.tensordot(q, k, ([2], [1])) * s["scale"]  # token, head, key
            pos = torch.arange(n - (hi - lo), n, device=DEV)[:, None, None]
            key = torch.arange(n, device=DEV)
            hidden = key > pos
            if s["window"]:
                hidden = hidden | (key <= pos - s["window"])
            score = score.masked_fill(hidden, -math.inf)
            z = torch.logsumexp(score, -1)
            lse[lo:hi, h * group:(h + 1) * group] = z
            out[lo:hi, h * group:(h + 1) * group] = torch.tensordot(torch.exp(score - z[..., None]), v, ([2], [0]))
    return [out, lse]


def _exact_logits(s):
    y = s["logits"].double()
    hist, bias = s["hist_start"].tolist(), s["bias_start"].tolist()
    vocab = y.shape[1]
    for i in range(y.shape[0]):
        tokens = s["history"][hist[i]:hist[i + 1]].long()
        n = int(s["prompt_len"][i])
        was = torch.bincount(tokens, minlength=vocab) > 0
        made = torch.bincount(tokens[n:], minlength=vocab).double()
        r = s["repetition"][i].double()
        row = y[i]
        row = torch.where(was & (row > 0), row / r, torch.where(was, row * r, row))
        row = row - made * s["frequency"][i].double() - (made > 0).double() * s["presence"][i].double()
        ids = s["bias_ids"][bias[i]:bias[i + 1]].long()
        row[ids] += s["bias_values"][bias[i]:bias[i + 1]].double()
        if s["allowed"] is not None:
            bits = (s["allowed"][i][:, None] >> torch.arange(32, device=DEV, dtype=torch.int32)) & 1
            row[bits.flatten()[:vocab] == 0] = -math.inf
        y[i] = row
    return [y]


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    s = prepare(case, seed)
    return {"append": _exact_append, "attn": _exact_attn, "logits": _exact_logits}[case["op"]](s)
