"""The operators of a mixture-of-experts layer over the 4-bit weights and cache, as measured cases.

  rope    queries rotated by their positions, keys rotated on their way into
          the paged Q4_0 cache, values appended beside them, both read back
  route   experts chosen for each token, their weights, and the (token, slot)
          pairs put in the order of their experts
  geglu   each pair's feed-forward input, gelu(x Wg^T) * (x Wu^T), with its
          expert's Q4_0 weights
  down    each token's weighted sum of its experts' down projections

Each has a plain form in elementary torch operations (fp32, one rounding at
the end; the choice of experts in 64 bits) and the library's own call; `own`
chooses between them.
"""
import math
import random
import zlib

import numpy as np
import torch

own = False

DEV = "cuda"


def _qmm():
    from block_quantized_matmul_gguf_gb300 import qmm
    return qmm


# ---- cases --------------------------------------------------------------------

def listed():
    return [
        # one decode step of sixteen requests: 8 query heads on 2 of 256, the
        # decode layer's own projections, far positions
        {"name": "rope-decode-16", "op": "rope", "tokens": 16, "heads": 8, "kv_heads": 2, "dim": 256, "rot": 256, "interleaved": False, "page": 64, "far": 131072, "dtype": "f32"},
        # a long prompt, an odd number of tokens, a part of each head rotated
        {"name": "rope-prompt-8191", "op": "rope", "tokens": 8191, "heads": 16, "kv_heads": 4, "dim": 128, "rot": 64, "interleaved": True, "page": 64, "far": 40000, "dtype": "bf16"},
        # the router of one request's next token: latency
        {"name": "route-one", "op": "route", "tokens": 1, "experts": 64, "topk": 8, "score": "softmax", "bias": False, "groups": 1, "kept": 1, "best": 1, "dtype": "f32"},
        # a batch of decoding requests with a bias that balances the experts
        {"name": "route-batch-128", "op": "route", "tokens": 128, "experts": 128, "topk": 8, "score": "softmax", "bias": True, "groups": 1, "kept": 1, "best": 1, "dtype": "f32"},
        # a chunk of prompts, sigmoid scores, groups of experts
        {"name": "route-prompt-8191", "op": "route", "tokens": 8191, "experts": 256, "topk": 8, "score": "sigmoid", "bias": True, "groups": 8, "kept": 4, "best": 2, "dtype": "f32"},
        # one request's next token: eight of 64 experts, the decode layer's
        # hidden size
        {"name": "geglu-one", "op": "geglu", "tokens": 1, "experts": 64, "topk": 8, "n": 1024, "k": 2048, "dtype": "f32"},
        # sixteen requests, one token each: most experts, a token or two each
        {"name": "geglu-batch-16", "op": "geglu", "tokens": 16, "experts": 64, "topk": 8, "n": 1024, "k": 2048, "dtype": "f32"},
        # a larger batch in bf16: some sixteen tokens an expert
        {"name": "geglu-batch-128", "op": "geglu", "tokens": 128, "experts": 64, "topk": 8, "n": 1024, "k": 2048, "dtype": "bf16"},
        # a chunk of prompts, an odd number of tokens: the tensor cores' case
        {"name": "geglu-prompt-2047", "op": "geglu", "tokens": 2047, "experts": 64, "topk": 8, "n": 1024, "k": 2048, "dtype": "bf16"},
        # the same requests' down projections
        {"name": "down-one", "op": "down", "tokens": 1, "experts": 64, "topk": 8, "n": 2048, "k": 1024, "dtype": "f32"},
        {"name": "down-batch-128", "op": "down", "tokens": 128, "experts": 64, "topk": 8, "n": 2048, "k": 1024, "dtype": "bf16"},
        {"name": "down-prompt-2047", "op": "down", "tokens": 2047, "experts": 64, "topk": 8, "n": 2048, "k": 1024, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "route", "geglu", "geglu", "down", "down"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "rope":
        kv, dim = rng.choice([1, 2, 4]), rng.choice([64, 128, 256])
        return {"op": op, "tokens": _log(rng, 1, 8191), "heads": kv * rng.choice([1, 2, 4]), "kv_heads": kv, "dim": dim,
                "rot": rng.choice([dim, dim // 2, dim // 4, dim - 24]), "interleaved": rng.choice([True, False]),
                "page": rng.choice([16, 32, 64, 128]), "far": _log(rng, 8191, 131072), "dtype": dtype}
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * _log(rng, 4, 256 // groups)
        kept = rng.randint(1, groups)
        best = rng.choice([1, 2])
        return {"op": op, "tokens": _log(rng, 1, 8191), "experts": experts,
                "topk": rng.randint(1, min(8, kept * experts // groups)), "score": rng.choice(["softmax", "sigmoid"]),
                "bias": rng.choice([True, False]), "groups": groups, "kept": kept, "best": best, "dtype": dtype}
    experts = rng.choice([8, 16, 60, 64, 128])
    topk = rng.randint(1, min(8, experts))
    wide, narrow = 32 * _log(rng, 8, 128), 32 * _log(rng, 4, 64)  # hidden size, expert width
    if rng.random() < 0.6:  # most models' sizes are multiples of 256
        wide, narrow = -(-wide // 256) * 256, -(-narrow // 256) * 256
    while experts * wide * narrow > 64 * 2048 * 1024:
        wide, narrow = max(256, wide // 64 * 32), max(128, narrow // 64 * 32)
    tokens = _log(rng, 1, 64) if dtype == "f32" else _log(rng, 1, 2047)
    tokens = max(1, min(tokens, 2047 * 8 * 2048 * 1024 // (topk * wide * narrow)))
    n, k = (narrow, wide) if op == "geglu" else (wide, narrow)
    return {"op": op, "tokens": tokens, "experts": experts, "topk": topk, "n": n, "k": k, "dtype": dtype}


def _key(case):
    return zlib.crc32(str(sorted((k, str(v)) for k, v in case.items() if k != "name")).encode())


def _choice(case):
    """Expert ids [tokens][topk] of each token, from the case alone: some experts are more popular than others."""
    r = np.random.default_rng(_key(case))
    popular = 0.5 * r.standard_normal(case["experts"])
    like = r.gumbel(size=(case["tokens"], case["experts"])) + popular
    return np.argsort(-like, axis=1, kind="stable")[:, :case["topk"]]


# ---- inputs --------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _weights(g, experts, n, k):
    """Random Q4_0 blocks [experts][n][k / 32 * 18]: scales as of trained weights, any codes."""
    blocks = torch.randint(0, 256, (experts, n, k // 32, 18), generator=g, device=DEV, dtype=torch.uint8)
    d = torch.rand(experts, n, k // 32, 1, generator=g, device=DEV) * 0.019 + 0.001
    blocks[..., :2] = d.half().view(torch.uint8)
    return blocks.flatten(2)


def _values(blocks):
    """The fp32 values [..., k] of Q4_0 blocks [..., k / 32 * 18]."""
    b = blocks.unflatten(-1, (-1, 18))
    d = b[..., :2].contiguous().view(torch.float16).float()
    q = b[..., 2:]
    return ((torch.cat([q & 15, q >> 4], -1).float() - 8) * d).flatten(-2)


def _quantize(x):
    """Q4_0 codes [..., D/2] and scales [..., D/32] of x [..., D] (fp32)."""
    b = x.unflatten(-1, (-1, 32))
    top, low = b.amax(-1), b.amin(-1)
    extreme = torch.where(top >= -low, top, low)
    d = (extreme / -8).clamp(-65504.0, 65504.0).half()
    f = d.float()[..., None]
    q = torch.where(f == 0, torch.full_like(b, 8.0), (torch.round(b / f) + 8).clamp(0, 15)).to(torch.uint8)
    return (q[..., :16] | (q[..., 16:] << 4)).flatten(-2), d


def _cached(codes, scales):
    """The fp32 values [..., D] that codes and scales stand for."""
    c = codes.unflatten(-1, (-1, 16))
    n = torch.cat([c & 15, c >> 4], -1).float() - 8
    return (n * scales.float()[..., None]).flatten(-2)


def prepare(case, seed):
    g = _gen(seed)
    s = {"op": case["op"], "case": case}
    if case["op"] == "rope":
        n, heads, kv, dim, page, rot = (case[k] for k in ("tokens", "heads", "kv_heads", "dim", "page", "rot"))
        pages = -(-n // page) + 5
        order = torch.randperm(pages, generator=g, device=DEV)
        token = torch.arange(n, device=DEV)
        # the cosines and sines of every position, made once, in 64 bits
        angle = torch.arange(case["far"], device=DEV, dtype=torch.float64)[:, None] * \
            10000.0 ** (torch.arange(rot // 2, device=DEV, dtype=torch.float64) * (-2.0 / rot))
        # q, k and v lie side by side in one projection's output
        both = torch.randn(n, heads + 2 * kv, dim, generator=g, device=DEV).to(_dtype(case))
        if n <= 64:  # single tokens of requests that have come far
            positions = torch.randint(0, case["far"], (n,), generator=g, device=DEV)
        else:
            positions = token + int(torch.randint(0, case["far"] - n + 1, (1,), generator=g, device=DEV))
        s.update(q=both[:, :heads], k=both[:, heads:heads + kv], v=both[:, heads + kv:],
                 slots=order[token // page] * page + token % page, positions=positions.int(),
                 table=torch.cat([angle.cos(), angle.sin()], 1).float().contiguous(),
                 codes=[torch.zeros(pages, kv, page, dim // 2, dtype=torch.uint8, device=DEV) for _ in range(2)],
                 scales=[torch.zeros(pages, kv, page, dim // 32, dtype=torch.float16, device=DEV) for _ in range(2)],
                 q_out=torch.empty(n, heads, dim, dtype=both.dtype, device=DEV),
                 out=[torch.empty(n, kv, dim, device=DEV) for _ in range(2)])
    elif case["op"] == "route":
        n, e, k = case["tokens"], case["experts"], case["topk"]
        popular = 0.5 * torch.randn(e, generator=g, device=DEV)
        s.update(logits=(torch.randn(n, e, generator=g, device=DEV) * 1.5 + popular).to(_dtype(case)),
                 bias=torch.randn(e, generator=g, device=DEV) * (0.2 if case["score"] == "sigmoid" else 0.01)
                 if case["bias"] else None, renormalize=True, scale=2.5 if case["score"] == "sigmoid" else 1.0,
                 ids=torch.empty(n, k, dtype=torch.int32, device=DEV), weights=torch.empty(n, k, device=DEV),
                 expert_start=torch.empty(e + 1, dtype=torch.int32, device=DEV),
                 pairs=torch.empty(n * k, dtype=torch.int32, device=DEV))
    else:
        t, e, topk, n, k = (case[x] for x in ("tokens", "experts", "topk", "n", "k"))
        ids = _choice(case)
        flat = ids.reshape(-1)
        counts = np.bincount(flat, minlength=e)
        active = np.flatnonzero(counts)
        s.update(ids=torch.from_numpy(ids).to(DEV).int(),
                 expert_start=torch.from_numpy(np.concatenate([[0], counts.cumsum()])).to(DEV).int(),
                 pairs=torch.from_numpy(np.argsort(flat, kind="stable")).to(DEV).int(),
                 active=torch.from_numpy(active).to(DEV), most=int(counts.max()),
                 weights=torch.softmax(torch.randn(t, topk, generator=g, device=DEV), -1))
        if case["op"] == "geglu":
            s.update(wg=_weights(g, e, n, k), wu=_weights(g, e, n, k),
                     x=torch.randn(t, k, generator=g, device=DEV).to(_dtype(case)),
                     h=torch.empty(t * topk, n, dtype=_dtype(case), device=DEV))
        else:
            # gated activations: many near nothing, some large
            h = torch.randn(t * topk, k, generator=g, device=DEV)
            h = torch.nn.functional.gelu(2 * h) * torch.randn(t * topk, k, generator=g, device=DEV)
            s.update(wd=_weights(g, e, n, k), h=h.to(_dtype(case)),
                     y=torch.empty(t, n, dtype=_dtype(case), device=DEV))
    if own:  # the handle and the workspaces that a program makes once
        if case["op"] == "rope":
            s["cache"] = _qmm().KvCacheQ4_0(s["codes"][0], s["scales"][0], s["codes"][1], s["scales"][1])
        if case["op"] == "route":
            s["workspace"] = _qmm().route_workspace(case["tokens"], case["experts"])
        if case["op"] == "down":
            s["workspace"] = _qmm().experts_workspace(case["tokens"], case["topk"], case["n"], case["k"])
    return s


# ---- one pass --------------------------------------------------------------------

def run(state):
    return (_own if own else _plain)[state["op"]](state)


def _own_rope(s):
    q = _qmm()
    q.qmm_kv_append_rope_q4_0(s["cache"], s["k"], s["v"], s["slots"], s["positions"], s["table"], q=s["q"],
                              q_out=s["q_out"], interleaved=s["case"]["interleaved"])
    q.qmm_kv_read_q4_0(s["cache"], s["slots"], s["out"][0], s["out"][1])
    return [s["q_out"], s["out"][0], s["out"][1]]


def _own_route(s):
    c = s["case"]
    _qmm().qmm_route(s["logits"], s["ids"], s["weights"], s["expert_start"], s["pairs"], bias=s["bias"],
                     score=c["score"], groups=c["groups"], group_topk=c["kept"], group_best=c["best"],
                     renormalize=s["renormalize"], scale=s["scale"], workspace=s["workspace"])
    return [s["ids"], s["weights"], s["expert_start"], s["pairs"]]


def _own_geglu(s):
    c = s["case"]
    _qmm().qmm_experts_geglu_q4_0(s["wg"], s["wu"], s["x"], s["h"], s["expert_start"], s["pairs"], c["topk"], c["n"],
                                  c["k"])
    return [s["h"]]


def _own_down(s):
    c = s["case"]
    _qmm().qmm_experts_down_q4_0(s["wd"], s["h"], s["y"], s["ids"], s["weights"], s["expert_start"], s["pairs"],
                                 c["n"], c["k"], workspace=s["workspace"])
    return [s["y"]]


_own = {"rope": _own_rope, "route": _own_route, "geglu": _own_geglu, "down": _own_down}


def _turned(x, c, s, interleaved):
    """x [n][heads][rot] rotated by cosines and sines [n][1][rot / 2], in fp32."""
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else x.chunk(2, -1)
    u, v = a * c - b * s, a * s + b * c
    return torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)


def _plain_rope(s):
    case = s["case"]
    rot, page = case["rot"], case["page"]
    c, d = s["table"][s["positions"].long()][:, None].chunk(2, -1)
    q, k = (torch.cat([_turned(x[..., :rot].float(), c, d, case["interleaved"]), x[..., rot:].float()], -1)
            for x in (s["q"], s["k"]))
    at, off = s["slots"] // page, s["slots"] % page
    kc, ks = _quantize(k)
    vc, vs = _quantize(s["v"].float())
    s["codes"][0][at, :, off], s["scales"][0][at, :, off] = kc, ks
    s["codes"][1][at, :, off], s["scales"][1][at, :, off] = vc, vs
    return [q.to(s["q"].dtype), _cached(s["codes"][0][at, :, off], s["scales"][0][at, :, off]),
            _cached(s["codes"][1][at, :, off], s["scales"][1][at, :, off])]


def _plain_route(s):
    c = s["case"]
    n, e = s["logits"].shape
    x = s["logits"].double()  # the choice in 64 bits: near scores keep their order
    score = torch.sigmoid(x)
    if c["score"] == "softmax":
        w = torch.exp(x - x.amax(-1, keepdim=True))
        score = w / w.sum(-1, keepdim=True)
    choice = score + s["bias"].double() if s["bias"] is not None else score
    if c["groups"] > 1:
        inside = choice.view(n, c["groups"], -1)
        best = inside.sort(-1, descending=True).values[..., :c["best"]].sum(-1)
        order = best.sort(dim=-1, descending=True, stable=True).indices[:, :c["kept"]]
        kept = torch.zeros_like(best, dtype=torch.bool).scatter(1, order, True)
        choice = inside.masked_fill(~kept[..., None], -math.inf).flatten(1)
    ids = choice.sort(dim=-1, descending=True, stable=True).indices[:, :c["topk"]]
    w = score.gather(1, ids)
    if s["renormalize"]:
        w = w / w.sum(-1, keepdim=True)
    flat = ids.reshape(-1)
    starts = (flat[None] < torch.arange(e + 1, device=DEV)[:, None]).sum(-1)
    return [ids.int(), (w * s["scale"]).float(), starts.int(), flat.sort(stable=True).indices.int()]


def _places(s, rows):
    """Padded places of the pairs by active expert: source rows [active][most], and what is real."""
    start = s["expert_start"].long()
    lo, hi = start[s["active"]], start[s["active"] + 1]
    at = lo[:, None] + torch.arange(s["most"], device=DEV)
    real = at < hi[:, None]
    at = at.clamp(max=rows - 1)
    return at, real


def _plain_geglu(s):
    rows = s["pairs"].numel()
    at, real = _places(s, rows)
    x = s["x"].float()[s["pairs"].long() // s["case"]["topk"]][at]  # [active][most][k]
    g = x @ _values(s["wg"][s["active"]]).transpose(1, 2)
    u = x @ _values(s["wu"][s["active"]]).transpose(1, 2)
    h = g / 2 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g))) * u
    return [h[real].to(s["x"].dtype)]  # in the order of the pairs


def _plain_down(s):
    rows = s["pairs"].numel()
    at, real = _places(s, rows)
    z = (s["h"].float()[at] @ _values(s["wd"][s["active"]]).transpose(1, 2))[real]
    z = torch.empty_like(z).index_copy_(0, s["pairs"].long(), z)
    t, topk = s["ids"].shape
    return [(z.view(t, topk, -1) * s["weights"][..., None]).sum(1).to(s["h"].dtype)]


_plain = {"rope": _plain_rope, "route": _plain_route, "geglu": _plain_geglu, "down": _plain_down}


# ---- what a pass cannot do without --------------------------------------------------

def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    n = case["tokens"]
    if case["op"] == "rope":
        q, kv = n * case["heads"] * case["dim"], n * case["kv_heads"] * case["dim"] * 2
        # inputs, rows of the table, slots twice, positions; q out, the cache written and read once, the values out
        return {"bytes": (2 * q + kv) * size + n * (4 * case["rot"] + 20) + 2 * kv * 18 // 32 + 4 * kv,
                "flops": 6 * (q + kv // 2) * case["rot"] // (2 * case["dim"]) + 4 * kv}
    if case["op"] == "route":
        e = case["experts"]
        return {"bytes": n * e * size + 12 * n * case["topk"] + 4 * (e + 1) + (4 * e if case["bias"] else 0), "flops": 6 * n * e}
    pairs, active = n * case["topk"], len(np.unique(_choice(case)))
    matrix = case["n"] * case["k"] * 18 // 32
    if case["op"] == "geglu":
        return {"bytes": 2 * active * matrix + n * case["k"] * size + pairs * (case["n"] * size + 4),
                "flops": 4 * pairs * case["n"] * case["k"]}
    return {"bytes": active * matrix + pairs * (case["k"] * size + 12) + n * case["n"] * size,
            "flops": 2 * pairs * case["n"] * case["k"]}


# ---- the definition, in 64 bits ------------------------------------------------------

def _exact_weights(blocks):
    """[n][k]: byte j of a block's codes holds value j in its low and value j + 16 in its high four bits."""
    n = blocks.shape[0]
    b = blocks.reshape(n, -1, 18)
    d = b[:, :, :2].contiguous().view(torch.float16).double()
    out = torch.empty(n, b.shape[1], 32, dtype=torch.float64, device=DEV)
    out[:, :, :16] = (b[:, :, 2:] % 16).double() - 8
    out[:, :, 16:] = torch.div(b[:, :, 2:], 16, rounding_mode="floor").double() - 8
    return (out * d).reshape(n, -1)


def _exact_cached(x):
    """What a block of 32 values becomes in the cache, from values in 64 bits."""
    b = x.unflatten(-1, (-1, 32))
    size, at = b.abs().max(-1)
    extreme = b.gather(-1, at[..., None])[..., 0]
    extreme = torch.where(b.amax(-1) == size, size, extreme)  # of +a and -a, the positive one
    d = (extreme / -8).clamp(-65504, 65504).half().double()[..., None]
    n = torch.where(d == 0, 0.0, torch.round(b / torch.where(d == 0, 1.0, d)).clamp(-8, 7))
    return (n * d).flatten(-2)


def _exact_rope(s):
    """Rotated keys are defined to the bit, because their codes are: each product and each sum in fp32, rounded once."""
    case = s["case"]
    rot = case["rot"]
    row = s["table"].double()[s["positions"].long()]
    c, d = row[:, None, :rot // 2], row[:, None, rot // 2:]

    def turned(x, fl):
        y = x.double().clone()
        first = slice(0, rot, 2) if case["interleaved"] else slice(0, rot // 2)
        second = slice(1, rot, 2) if case["interleaved"] else slice(rot // 2, rot)
        a, b = y[..., first].clone(), y[..., second].clone()
        y[..., first], y[..., second] = fl(fl(a * c) - fl(b * d)), fl(fl(a * d) + fl(b * c))
        return y

    return [turned(s["q"], lambda v: v), _exact_cached(turned(s["k"], lambda v: v.float().double())),
            _exact_cached(s["v"].double())]


def _exact_route(s):
    """Weights of the ids; the ids and the order are whole numbers."""
    c = s["case"]
    x = s["logits"].double().cpu().numpy()
    score = 1 / (1 + np.exp(-x)) if c["score"] == "sigmoid" else None
    if score is None:
        score = np.exp(x - np.logaddexp.reduce(x, axis=1)[:, None])
    value = score + (s["bias"].double().cpu().numpy() if s["bias"] is not None else 0.0)
    if c["groups"] > 1:
        inside = value.reshape(len(x), c["groups"], -1)
        best = np.partition(inside, inside.shape[2] - min(c["best"], inside.shape[2]), axis=2)
        best = best[:, :, -c["best"]:].sum(2)
        rank = np.argsort(np.argsort(-best, axis=1, kind="stable"), axis=1)
        value = np.where((rank < c["kept"])[:, :, None], inside, -np.inf).reshape(len(x), -1)
    ids = np.argsort(-value, axis=1, kind="stable")[:, :c["topk"]]
    w = np.take_along_axis(score, ids, 1)
    w = w / w.sum(1, keepdims=True) * s["scale"]
    return [None, torch.from_numpy(w).to(DEV), None, None]


def _exact_geglu(s):
    starts, topk = s["expert_start"].tolist(), s["case"]["topk"]
    x = s["x"].double()
    h = torch.empty(s["h"].shape, dtype=torch.float64, device=DEV)
    for e in range(len(starts) - 1):
        lo, hi = starts[e], starts[e + 1]
        if lo < hi:
            rows = x[torch.div(s["pairs"][lo:hi].long(), topk, rounding_mode="floor")]
            g, u = (torch.einsum("rk,nk->rn", rows, _exact_weights(w[e])) for w in (s["wg"], s["wu"]))
            a = math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
            h[lo:hi] = g * torch.sigmoid(2 * a) * u  # the same function as with the tanh
    return [h]


def _exact_down(s):
    starts = s["expert_start"].tolist()
    t, topk = s["ids"].shape
    y = torch.zeros(t, s["case"]["n"], dtype=torch.float64, device=DEV)
    w = s["weights"].double().flatten()
    for e in range(len(starts) - 1):
        lo, hi = starts[e], starts[e + 1]
        if lo < hi:
            at = s["pairs"][lo:hi].long()
            z = torch.einsum("rk,nk->rn", s["h"][lo:hi].double(), _exact_weights(s["wd"][e]))
            y.index_add_(0, torch.div(at, topk, rounding_mode="floor"), z * w[at][:, None])
    return [y]


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "route": _exact_route, "geglu": _exact_geglu, "down": _exact_down}[case["op"]](s)
