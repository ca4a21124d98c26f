"""The experts' products against 64 bits, within bounds derived from their
roundings (experts_ref), and within a norm that random signs allow."""
import numpy as np
import pytest

import experts_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def qmm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_quantized_matmul_gguf_gb300 import build, qmm
    build.build_library()
    return qmm


def choice(rng, tokens, experts, topk, kind="any"):
    """ids [tokens][topk]: any experts, always the same ones, or with tokens that are not there."""
    if kind == "same":
        return np.tile(rng.permutation(experts)[:topk], (tokens, 1))
    ids = np.argsort(rng.random((tokens, experts)), axis=1)[:, :topk]
    if kind == "padded":
        ids[tokens - tokens // 3:] = -1
    return ids


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def near(got, want, limit, exact, rows=slice(None)):
    got, want, limit = got.double().cpu().numpy()[rows], want[rows], limit[rows]
    assert np.isfinite(got).all()
    bad = np.abs(got - want) > limit
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])
    # roundings of random sign: a few of bf16's half steps in all, or of 2^-18
    size = np.linalg.norm(want)
    if want.size >= 256:
        assert np.linalg.norm(got - want) <= (2.0 ** -18 if exact else 4 * 2.0 ** -8) * size


def run_geglu(qmm, rng, tokens, experts, topk, n, k, x_type=F32, h_type=F32, kind="any"):
    ids = choice(rng, tokens, experts, topk, kind)
    starts, pairs = ref.plan_of(ids, experts)
    bg, bu = ref.blocks(rng, experts, n, k), ref.blocks(rng, experts, n, k)
    x = torch.from_numpy(rng.standard_normal((tokens, k)).astype(np.float32)).to(x_type)
    h = torch.full((tokens * topk, n), 7.0, dtype=h_type, device="cuda")
    args = (dev(bg), dev(bu), x.cuda(), h, dev(starts), dev(pairs), topk, n, k)
    qmm.qmm_experts_geglu_q4_0(*args)
    want, limit = ref.experts_geglu(x.double().numpy(), bg, bu, starts, pairs, topk, h_type is F32, x_type is F32)
    real = starts[-1]
    near(h, want, limit, h_type is F32, slice(0, real))
    assert (h[real:] == 7.0).all()  # rows of no pair
    again = torch.full_like(h, 7.0)
    qmm.qmm_experts_geglu_q4_0(*args[:3], again, *args[4:])
    assert torch.equal(again, h)
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


def run_down(qmm, rng, tokens, experts, topk, n, k, h_type=F32, y_type=F32, kind="any"):
    ids = choice(rng, tokens, experts, topk, kind)
    starts, pairs = ref.plan_of(ids, experts)
    bd = ref.blocks(rng, experts, n, k)
    h = torch.from_numpy(rng.standard_normal((tokens * topk, k)).astype(np.float32)).to(h_type)
    weights = rng.random((tokens, topk)).astype(np.float32)
    y = torch.full((tokens, n), 7.0, dtype=y_type, device="cuda")
    args = (dev(bd), h.cuda(), y, dev(ids.astype(np.int32)), dev(weights), dev(starts), dev(pairs), n, k)
    qmm.qmm_experts_down_q4_0(*args)
    want, limit = ref.experts_down(h.double().numpy(), bd, ids, weights, starts, pairs, y_type is F32, h_type is F32)
    near(y, want, limit, y_type is F32)
    again = torch.full_like(y, 7.0)
    qmm.qmm_experts_down_q4_0(*args[:2], again, *args[3:], workspace=qmm.experts_workspace(tokens, topk, n, k))
    assert torch.equal(again, y)
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


SIZES = [  # tokens, experts, topk, n, k
    (1, 1, 1, 1, 32), (1, 4, 2, 16, 256), (3, 5, 5, 33, 64), (2, 8, 3, 100, 512), (7, 3, 2, 48, 288), (9, 16, 4, 130, 96),
    (16, 8, 2, 64, 1024), (31, 6, 3, 20, 800), (5, 4, 2, 96, 2048), (4, 3, 3, 40, 4096), (3, 2, 2, 33, 8192),
    (2, 64, 4, 130, 512), (2, 40, 8, 70, 2048), (1, 64, 8, 300, 4096),
]
LONG = [(70, 4, 2, 40, 256), (130, 3, 2, 64, 512), (300, 8, 4, 260, 256), (513, 2, 1, 136, 512), (257, 16, 8, 64, 288), (20, 96, 2, 100, 512), (90, 5, 2, 150, 32),
        (140, 3, 1, 70, 992), (200, 6, 3, 129, 2080), (60, 16, 4, 256, 480)]
TYPES = [(F32, F32), (BF16, BF16), (BF16, F32), (F32, BF16)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("types", TYPES, ids=str)
def test_geglu(qmm, size, types):
    run_geglu(qmm, np.random.default_rng(sum(size)), *size, *types)


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("types", TYPES, ids=str)
def test_down(qmm, size, types):
    run_down(qmm, np.random.default_rng(sum(size)), *size, *types)


@pytest.mark.parametrize("size", LONG)
@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("kind", ["any", "same", "padded"])
def test_many_tokens(qmm, size, types, kind):
    rng = np.random.default_rng(sum(size))
    run_geglu(qmm, rng, *size, *types, kind=kind)
    run_down(qmm, rng, *size, *types, kind=kind)


@pytest.mark.parametrize("types", TYPES, ids=str)
def test_more_experts_than_threads(qmm, types):
    rng = np.random.default_rng(5)
    run_geglu(qmm, rng, 9, 1024, 32, 16, 32, *types)
    run_down(qmm, rng, 9, 1024, 32, 24, 32, *types)


@pytest.mark.parametrize("k", [32, 256, 288, 1024])
@pytest.mark.parametrize("tokens", [5, 40, 200])
def test_each_weight_alone(qmm, k, tokens):
    """One-hot rows: the products are the weights themselves, exactly (fp32), or rounded once or twice (bf16)."""
    rng = np.random.default_rng(k)
    experts, n = 3, 50
    bd = ref.blocks(rng, experts, n, k)
    w, _ = ref.matrix(bd)
    ids = rng.integers(0, experts, (tokens, 1))
    starts, pairs = ref.plan_of(ids, experts)
    at = rng.integers(0, k, tokens)
    h = np.zeros((tokens, k), dtype=np.float32)
    h[np.arange(tokens), at] = 1.0
    h = h[pairs]  # in the order of the pairs
    want = w[ids[:, 0], :, at]
    ones = np.ones((tokens, 1), dtype=np.float32)
    for h_type, y_type in TYPES:
        y = torch.empty(tokens, n, dtype=y_type, device="cuda")
        qmm.qmm_experts_down_q4_0(dev(bd), dev(h, h_type), y, dev(ids.astype(np.int32)), dev(ones), dev(starts), dev(pairs), n, k)
        got = y.double().cpu().numpy()
        if y_type is F32:
            assert np.array_equal(got, want)
        else:  # one rounding of the weight or of the result, or both
            assert (np.abs(got - want) <= 2.1 * 2.0 ** -8 * np.abs(want) + 2.0 ** -12 * 16 * 0.02).all()


@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("tokens", [6, 150])
def test_rows_keep_to_themselves(qmm, types, tokens):
    """A row without a number, a huge and a tiny one beside ordinary ones."""
    rng = np.random.default_rng(11)
    experts, topk, n, k = 2, 1, 40, 512
    ids = np.zeros((tokens, 1), dtype=np.int64)
    ids[tokens // 2:] = 1
    starts, pairs = ref.plan_of(ids, experts)
    bg, bu = ref.blocks(rng, experts, n, k), ref.blocks(rng, experts, n, k)
    x = rng.standard_normal((tokens, k)).astype(np.float32)
    x[2] *= 1e-20
    x[3] *= 1e9
    x = torch.from_numpy(x).to(types[0])
    h = [torch.empty(tokens, n, dtype=types[1], device="cuda") for _ in range(2)]
    rest = (dev(starts), dev(pairs), topk, n, k)
    qmm.qmm_experts_geglu_q4_0(dev(bg), dev(bu), x.cuda(), h[0], *rest)
    want, limit = ref.experts_geglu(x.double().numpy(), bg, bu, starts, pairs, topk, types[1] is F32, types[0] is F32)
    ordinary = [i for i in range(tokens) if i not in (2, 3)]
    got = h[0].double().cpu().numpy()
    assert (np.abs(got - want) <= limit)[ordinary + [3]].all()
    assert (np.abs(got[2] - want[2]) <= limit[2] + 1e-37).all()
    x[1, 5], x[4, 300] = float("nan"), float("inf")
    qmm.qmm_experts_geglu_q4_0(dev(bg), dev(bu), x.cuda(), h[1], *rest)
    keep = [i for i in range(tokens) if i not in (1, 4)]
    assert torch.equal(h[0][keep], h[1][keep])
    assert torch.isnan(h[1][1]).all() and not torch.isfinite(h[1][4]).any()


@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("off", [1, 3, 4])
@pytest.mark.parametrize("tokens", [6, 140])
def test_strides_and_alignment(qmm, types, off, tokens):
    rng = np.random.default_rng(off)
    experts, topk, n, k = 4, 2, 48, 256
    ids = choice(rng, tokens, experts, topk)
    starts, pairs = ref.plan_of(ids, experts)
    bg, bu, bd = (ref.blocks(rng, experts, *s) for s in ((n, k), (n, k), (k, 64)))
    x = torch.from_numpy(rng.standard_normal((tokens, k + off + 2)).astype(np.float32)).to(types[0]).cuda()[:, off:off + k]
    room = torch.full((tokens * topk, n + off + 1), 7.0, dtype=types[1], device="cuda")
    h = room[:, off:off + n]
    qmm.qmm_experts_geglu_q4_0(dev(bg), dev(bu), x, h, dev(starts), dev(pairs), topk, n, k)
    want, limit = ref.experts_geglu(x.double().cpu().numpy(), bg, bu, starts, pairs, topk, types[1] is F32, types[0] is F32)
    near(h, want, limit, types[1] is F32)
    assert (room[:, :off] == 7.0).all() and (room[:, off + n:] == 7.0).all()
    h = torch.from_numpy(rng.standard_normal((tokens * topk, 64 + off)).astype(np.float32)).to(types[0]).cuda()[:, off:]
    room = torch.full((tokens, k + off + 1), 7.0, dtype=types[1], device="cuda")
    y = room[:, off:off + k]
    weights = rng.random((tokens, topk)).astype(np.float32)
    qmm.qmm_experts_down_q4_0(dev(bd), h, y, dev(ids.astype(np.int32)), dev(weights), dev(starts), dev(pairs), k, 64)
    want, limit = ref.experts_down(h.double().cpu().numpy(), bd, ids, weights, starts, pairs, types[1] is F32, types[0] is F32)
    near(y, want, limit, types[1] is F32)
    assert (room[:, :off] == 7.0).all() and (room[:, off + k:] == 7.0).all()


@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16)], ids=str)
@pytest.mark.parametrize("tokens", [4, 200])
def test_a_layer_in_a_graph(qmm, types, tokens):
    """Routing and both products on a side stream, captured and replayed for other tokens and fewer of them."""
    rng = np.random.default_rng(8)
    experts, topk, hidden, width = 8, 3, 256, 96
    bg, bu, bd = (ref.blocks(rng, experts, *s) for s in ((width, hidden), (width, hidden), (hidden, width)))
    wg, wu, wd = dev(bg), dev(bu), dev(bd)
    i32 = dict(dtype=torch.int32, device="cuda")
    x = torch.empty(tokens, hidden, dtype=types[0], device="cuda")
    logits = torch.empty(tokens, experts, device="cuda")
    count = torch.empty(1, **i32)
    ids, weights = torch.empty(tokens, topk, **i32), torch.empty(tokens, topk, device="cuda")
    starts, pairs = torch.empty(experts + 1, **i32), torch.empty(tokens * topk, **i32)
    h = torch.empty(tokens * topk, width, dtype=types[0], device="cuda")
    y = torch.empty(tokens, hidden, dtype=types[1], device="cuda")
    ws, rs = qmm.experts_workspace(tokens, topk, hidden, width), qmm.route_workspace(tokens, experts)

    def fill(n):
        x.copy_(torch.from_numpy(rng.standard_normal((tokens, hidden)).astype(np.float32)))
        logits.copy_(torch.from_numpy(rng.standard_normal((tokens, experts)).astype(np.float32)))
        count.fill_(n)

    def layer():
        qmm.qmm_route(logits, ids, weights, starts, pairs, count=count, workspace=rs)
        qmm.qmm_experts_geglu_q4_0(wg, wu, x, h, starts, pairs, topk, width, hidden)
        qmm.qmm_experts_down_q4_0(wd, h, y, ids, weights, starts, pairs, hidden, width, workspace=ws)

    side = torch.cuda.Stream()
    fill(tokens)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        layer()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        layer()
    for n in (tokens, tokens - 1, 0):
        fill(n)
        graph.replay()
        torch.cuda.synchronize()
        r = ref.route(logits.double().cpu().numpy(), None, topk, "softmax", count=n)
        assert np.array_equal(ids.cpu().numpy(), r[0]) and np.array_equal(pairs.cpu().numpy(), r[3])
        exact = types[1] is F32
        want, limit = ref.experts_geglu(x.double().cpu().numpy(), bg, bu, r[2], r[3], topk, exact, types[0] is F32)
        near(h, want, limit, exact, slice(0, n * topk))
        want, limit = ref.experts_down(h.double().cpu().numpy(), bd, r[0], weights.cpu().numpy(), r[2], r[3], exact, types[0] is F32)
        near(y, want, limit, exact)
        assert (y[n:] == 0).all()
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16)], ids=str)
@pytest.mark.parametrize("tokens", [5, 150])
def test_bad_plans_are_recorded(qmm, types, tokens):
    rng = np.random.default_rng(3)
    experts, topk, n, k = 4, 2, 32, 256
    ids = choice(rng, tokens, experts, topk)
    starts, pairs = ref.plan_of(ids, experts)
    bg, bu = ref.blocks(rng, experts, n, k), ref.blocks(rng, experts, n, k)
    x = torch.from_numpy(rng.standard_normal((tokens, k)).astype(np.float32)).to(types[0])
    want, limit = ref.experts_geglu(x.double().numpy(), bg, bu, starts, pairs, topk, types[1] is F32, types[0] is F32)

    def run(starts, pairs):
        h = torch.full((tokens * topk, n), 7.0, dtype=types[1], device="cuda")
        qmm.qmm_experts_geglu_q4_0(dev(bg), dev(bu), x.cuda(), h, dev(starts), dev(pairs), topk, n, k)
        assert qmm.qmm_get_device_error() == qmm.QMM_ERR_INDEX
        return h

    for bad in (tokens * topk, -1, 1 << 30):  # a pair that is not there
        odd = pairs.copy()
        odd[1] = bad
        h = run(starts, odd)
        keep = np.arange(tokens * topk) != 1
        near(h, want, limit, types[1] is F32, keep)
        assert (h[1] == 7.0).all()
    for bad in (tokens * topk + 1, -3):  # a start outside: the experts on both sides of it are left out
        odd = starts.copy()
        odd[2] = bad
        h = run(odd, pairs)
        keep = np.r_[0:starts[1], starts[3]:starts[4]]
        near(h, want, limit, types[1] is F32, keep)
        assert (h[starts[1]:starts[3]] == 7.0).all()


def test_offsets_past_32_bits(qmm):
    """Weights of 2.4 GB: the last expert's rows lie past 2^31 bytes."""
    experts, n, k = 512, 1024, 8192
    wd = torch.zeros(experts, n, k // 32 * 18, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(1)
    last = ref.blocks(rng, n, k)
    wd[-1].copy_(dev(last))
    for tokens, types in ((3, (F32, F32)), (3, (BF16, BF16)), (90, (BF16, BF16))):
        ids = np.full((tokens, 1), experts - 1)
        starts, pairs = ref.plan_of(ids, experts)
        h = torch.from_numpy(rng.standard_normal((tokens, k)).astype(np.float32)).to(types[0])
        y = torch.empty(tokens, n, dtype=types[1], device="cuda")
        ones = np.ones((tokens, 1), dtype=np.float32)
        qmm.qmm_experts_down_q4_0(wd, h.cuda(), y, dev(ids.astype(np.int32)), dev(ones), dev(starts), dev(pairs), n, k)
        z, limit = ref.product(h.double().numpy(), last, types[1] is F32, types[0] is F32)
        near(y, z, limit + np.abs(z) * (2.0 ** -20 if types[1] is F32 else 2.1 * 2.0 ** -8), types[1] is F32)


def test_refusals(qmm):
    rng = np.random.default_rng(2)
    wg = dev(ref.blocks(rng, 2, 32, 64))
    i32 = dict(dtype=torch.int32, device="cuda")
    x, h = torch.zeros(3, 64, device="cuda"), torch.zeros(6, 32, device="cuda")
    starts, pairs = torch.zeros(3, **i32), torch.zeros(6, **i32)
    ids, weights = torch.zeros(3, 2, **i32), torch.zeros(3, 2, device="cuda")
    good = dict(wg=wg, wu=wg, x=x, h=h, expert_start=starts, pairs=pairs, topk=2, n=32, k=64)
    qmm.qmm_experts_geglu_q4_0(**good)
    for bad in (dict(x=x.half()), dict(x=x[:, :32]), dict(h=h[:5]), dict(pairs=pairs[:4]), dict(topk=3), dict(wg=wg[:1]),
                dict(x=x.cpu()), dict(pairs=pairs.long())):
        with pytest.raises(ValueError):
            qmm.qmm_experts_geglu_q4_0(**{**good, **bad})
    shifted = torch.zeros(wg.numel() + 2, dtype=torch.uint8, device="cuda")[2:]
    with pytest.raises(qmm.QmmError):
        qmm.qmm_experts_geglu_q4_0(**{**good, "wg": shifted})
    both = torch.zeros(9, 64, device="cuda")
    with pytest.raises(qmm.QmmError):  # h over x
        qmm.qmm_experts_geglu_q4_0(**{**good, "x": both[:3], "h": both[2:8, :32]})
    y = torch.zeros(3, 32, device="cuda")
    hd = torch.zeros(6, 64, device="cuda")
    good = dict(wd=wg, h=hd, y=y, ids=ids, weights=weights, expert_start=starts, pairs=pairs, n=32, k=64)
    qmm.qmm_experts_down_q4_0(**good)
    for bad in (dict(h=hd[:5]), dict(y=y[:2]), dict(weights=weights[:2]), dict(y=y.half()), dict(ids=ids.long())):
        with pytest.raises(ValueError):
            qmm.qmm_experts_down_q4_0(**{**good, **bad})
    with pytest.raises(qmm.QmmError):
        qmm.qmm_experts_down_q4_0(**{**good, "workspace": torch.empty(64, dtype=torch.uint8, device="cuda")})
    # nothing to do
    none = torch.zeros(0, 64, device="cuda")
    qmm.qmm_experts_geglu_q4_0(wg, wg, none, torch.zeros(0, 32, device="cuda"), starts, pairs[:0], 2, 32, 64)
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("k", [65536, 65568])
def test_long_rows(qmm, types, k):
    rng = np.random.default_rng(k)
    run_geglu(qmm, rng, 3, 3, 2, 20, k, *types)
    run_down(qmm, rng, 3, 3, 2, 20, k, *types)


@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16)], ids=str)
@pytest.mark.parametrize("k", [2048, 2080])
@pytest.mark.parametrize("tokens", [3, 1100])
def test_rows_far_apart_of_the_last_expert(qmm, types, k, tokens):
    """The last of 1024 experts of 5 GB of weights, rows of x and h 2^21 elements apart."""
    experts, n = 1024, 4352
    rng = np.random.default_rng(k + tokens)
    row = k // 32 * 18
    w = [torch.zeros((experts, n, row), dtype=torch.uint8, device="cuda") for _ in range(2)]
    assert w[0].numel() > 1 << 32
    last = [ref.blocks(rng, 1, n, k) for _ in w]
    for t, b in zip(w, last):
        t[-1] = dev(b[0])
    ids = np.full((tokens, 1), experts - 1)
    starts, pairs = ref.plan_of(ids, experts)
    apart = 1 << 21
    x = rng.standard_normal((tokens, k)).astype(np.float32)
    wide = torch.zeros((tokens, apart), dtype=types[0], device="cuda")[:, :k]
    wide.copy_(torch.from_numpy(x))
    some = [0, tokens // 2, tokens - 1]
    want, limit = ref.geglu(wide[some].double().cpu().numpy(), last[0][0], last[1][0], types[1] is F32, types[0] is F32)
    h = torch.zeros((tokens, apart), dtype=types[1], device="cuda")[:, :n]
    qmm.qmm_experts_geglu_q4_0(w[0], w[1], wide, h, dev(starts), dev(pairs), 1, n, k)
    near(h[some], want, limit, types[1] is F32)
    del h
    y = torch.zeros((tokens, apart), dtype=types[1], device="cuda")[:, :n]
    ones = torch.ones((tokens, 1), device="cuda")
    qmm.qmm_experts_down_q4_0(w[0], wide, y, dev(ids.astype(np.int32)), ones, dev(starts), dev(pairs), n, k)
    local, order = ref.plan_of(np.zeros((3, 1), dtype=np.int64), 1)
    want, limit = ref.experts_down(wide[some].double().cpu().numpy(), last[0], np.zeros((3, 1), dtype=np.int64),
                                   np.ones((3, 1)), local, order, types[1] is F32, types[0] is F32)
    near(y[some], want, limit, types[1] is F32)
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


def test_two_streams_at_once(qmm):
    """Calls that overlap, each with a workspace of its own, give what they give alone."""
    rng = np.random.default_rng(77)
    tokens, experts, topk, n, k = 300, 8, 2, 512, 1024
    cases = []
    for _ in range(2):
        ids = choice(rng, tokens, experts, topk)
        starts, pairs = ref.plan_of(ids, experts)
        x = dev(rng.standard_normal((tokens, k)).astype(np.float32), BF16)
        cases.append((dev(ref.blocks(rng, experts, n, k)), dev(ref.blocks(rng, experts, n, k)), dev(ref.blocks(rng, experts, k, n)),
                      x, dev(ids.astype(np.int32)), dev(rng.random((tokens, topk)).astype(np.float32)), dev(starts), dev(pairs)))

    def layer(c, stream=None):
        wg, wu, wd, x, ids, weights, starts, pairs = c
        h = torch.empty((tokens * topk, n), dtype=BF16, device="cuda")
        y = torch.empty((tokens, k), dtype=BF16, device="cuda")
        for _ in range(20):
            qmm.qmm_experts_geglu_q4_0(wg, wu, x, h, starts, pairs, topk, n, k, stream=stream)
            qmm.qmm_experts_down_q4_0(wd, h, y, ids, weights, starts, pairs, k, n, stream=stream)
        return y

    alone = [layer(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    both = []
    for c, s in zip(cases, streams):
        with torch.cuda.stream(s):
            both.append(layer(c))
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        assert torch.equal(a, b)


def test_plans_and_weights_written_just_before(qmm):
    """Calls back to back, each with a plan and weights that the stream writes right before it."""
    rng = np.random.default_rng(91)
    tokens, experts, topk, n, k = 64, 16, 2, 256, 512
    x = dev(rng.standard_normal((tokens, k)).astype(np.float32), BF16)
    sets = []
    for kind in ("any", "same", "padded", "any"):
        ids = choice(rng, tokens, experts, topk, kind)
        starts, pairs = ref.plan_of(ids, experts)
        sets.append((dev(ref.blocks(rng, experts, n, k)), dev(ref.blocks(rng, experts, n, k)), dev(starts), dev(pairs)))
    ws = qmm.experts_workspace(tokens, topk, n, k)
    want = []
    for wg, wu, starts, pairs in sets:
        h = torch.zeros((tokens * topk, n), dtype=BF16, device="cuda")
        qmm.qmm_experts_geglu_q4_0(wg, wu, x, h, starts, pairs, topk, n, k, workspace=ws)
        torch.cuda.synchronize()
        want.append(h)
    live = [torch.empty_like(t) for t in sets[0]]
    got = [torch.zeros_like(h) for h in want]
    for _ in range(50):
        for s, h in zip(sets, got):
            h.zero_()
            for to, t in zip(live, s):
                to.copy_(t)
            qmm.qmm_experts_geglu_q4_0(live[0], live[1], x, h, live[2], live[3], topk, n, k, workspace=ws)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16)], ids=str)
@pytest.mark.parametrize("k", [256, 288])
def test_a_plan_with_more_than_its_pairs_is_not_worked(qmm, types, k):
    """Starts 0, P, 0, P ..: every other expert claims all pairs."""
    tokens, experts, topk, n = 200, 64, 2, 64
    rng = np.random.default_rng(5)
    pairs = np.arange(tokens * topk, dtype=np.int32)
    starts = np.array([0, tokens * topk] * (experts // 2) + [0], dtype=np.int32)
    x = torch.from_numpy(rng.standard_normal((tokens, k)).astype(np.float32)).to(types[0]).cuda()
    b = dev(ref.blocks(rng, experts, n, k))
    h = torch.full((tokens * topk, n), 7.0, dtype=types[1], device="cuda")
    qmm.qmm_experts_geglu_q4_0(b, b, x, h, dev(starts), dev(pairs), topk, n, k)
    assert qmm.qmm_get_device_error() == qmm.QMM_ERR_INDEX
    assert (h == 7.0).all()
    # the same call of a sound plan, right behind it
    ids = choice(rng, tokens, experts, topk)
    starts, pairs = ref.plan_of(ids, experts)
    qmm.qmm_experts_geglu_q4_0(b, b, x, h, dev(starts), dev(pairs), topk, n, k)
    assert qmm.qmm_get_device_error() == qmm.QMM_OK
    assert (h != 7.0).any()
