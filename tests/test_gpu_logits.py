"""qmm_logits_adjust on the GPU against a plain 64-bit reference.

Bound: one division or product, one product, two sums, each rounded once:
|y - ref| <= 4 * 2^-24 * (|x * r| + |x / r| + c * freq + pres + sum |bias|) + 1e-37."""
import numpy as np
import pytest

import serving_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qmm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_quantized_matmul_gguf_gb300 import build, qmm as q
    build.build_library()
    q.load()
    q.qmm_get_device_error()
    return q


def ragged(lists, dtype):
    ends = np.concatenate([[0], np.cumsum([len(x) for x in lists])])
    flat = np.concatenate([np.asarray(x) for x in lists]) if lists else np.zeros(0)
    return torch.from_numpy(flat.astype(dtype)).cuda(), torch.from_numpy(ends.astype(np.int32)).cuda()


def pack(allowed):
    rows, vocab = allowed.shape
    words = np.zeros((rows, -(-vocab // 32) * 32), np.uint32)
    words[:, :vocab] = allowed
    w = (words.reshape(rows, -1, 32) << np.arange(32, dtype=np.uint32)).sum(-1, dtype=np.uint32)
    return torch.from_numpy(w.view(np.int32)).cuda()


def make(rng, rows, vocab, hist, nb, ids=None):
    x = (rng.standard_normal((rows, vocab)) * 3).astype(np.float32)
    h = [rng.integers(-3, vocab + 3, rng.integers(0, hist + 1)) if ids is None else
         rng.choice(ids, rng.integers(0, hist + 1)) for _ in range(rows)]
    prompt = np.array([rng.integers(0, len(a) + 2) for a in h])
    rep = 1 + rng.random(rows).astype(np.float32)
    freq, pres = rng.random(rows).astype(np.float32), rng.random(rows).astype(np.float32)
    bias = [[(int(t), float(np.float32(v))) for t, v in zip(rng.integers(-2, vocab + 2, nb), rng.standard_normal(nb))]
            for _ in range(rows)]
    return x, h, prompt, rep, freq, pres, bias, rng.random((rows, vocab)) < 0.5


def call(qmm, x, h, prompt, rep, freq, pres, bias, allowed, out=None, **leave):
    history, hist_start = ragged(h, np.int32)
    ids, start = ragged([[t for t, _ in b] for b in bias], np.int32)
    vals, _ = ragged([[v for _, v in b] for b in bias], np.float32)
    xd = torch.from_numpy(x).cuda() if isinstance(x, np.ndarray) else x
    out = torch.full_like(xd, 9.0) if out is None else out
    f = lambda a: torch.from_numpy(np.asarray(a, np.float32)).cuda()  # noqa: E731
    kw = dict(history=history, hist_start=hist_start, prompt_len=torch.from_numpy(prompt.astype(np.int32)).cuda(),
              repetition=f(rep), frequency=f(freq), presence=f(pres), bias_ids=ids, bias_values=vals,
              bias_start=start, allowed=None if allowed is None else pack(allowed))
    kw.update(leave)
    qmm.qmm_logits_adjust(xd, out, **kw)
    return out


def check(y, x, h, prompt, rep, freq, pres, bias, allowed):
    want = ref.logits(x, h, prompt, rep, freq, pres, bias, allowed)
    y = y.cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isneginf(y), np.isneginf(want))
    size = np.abs(x) * (rep[:, None] + 1 / rep[:, None]).astype(np.float64)
    for i in range(len(h)):
        ids = h[i][(h[i] >= 0) & (h[i] < x.shape[1])]
        c = np.bincount(ids, minlength=x.shape[1])
        size[i] += c * freq[i] + pres[i]
        for t, v in bias[i]:
            if 0 <= t < x.shape[1]:
                size[i, t] += abs(v)
    live = np.isfinite(want)
    assert (np.abs(y[live] - want[live]) <= 4 * 2.0 ** -24 * size[live] + 1e-37).all()


@pytest.mark.parametrize("rows,vocab,hist,nb", [
    (1, 1, 3, 1), (1, 31, 0, 0), (2, 32, 9, 4), (3, 33, 200, 70), (5, 1000, 50, 33), (1, 262144, 500, 10),
    (4, 32003, 3000, 64), (17, 8191, 1, 1), (70, 4097, 100, 5), (300, 2048, 40, 3), (64, 50001, 5000, 100),
])
def test_against_reference(qmm, rows, vocab, hist, nb):
    case = make(np.random.default_rng(rows * 31 + vocab), rows, vocab, hist, nb)
    y = call(qmm, *case)
    check(y, *case)
    assert torch.equal(y, call(qmm, *case))  # no order of atomics shows
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


@pytest.mark.parametrize("off_in,off_out,extra", [(0, 0, 1), (1, 1, 0), (2, 3, 2), (3, 0, 5), (0, 2, 4)])
def test_strides_and_alignments(qmm, off_in, off_out, extra):
    rows, vocab = 5, 3001
    case = make(np.random.default_rng(5), rows, vocab, 60, 9)
    size = rows * (vocab + extra) + 8
    rows_of = lambda t, off: torch.as_strided(t, (rows, vocab), (vocab + extra, 1), off)  # noqa: E731
    a = torch.full((size,), 3.0)
    rows_of(a, off_in).copy_(torch.from_numpy(case[0]))
    a, b = a.cuda(), torch.full((size,), 3.0).cuda()
    call(qmm, rows_of(a, off_in), *case[1:], out=rows_of(b, off_out))
    b = b.cpu()
    check(rows_of(b, off_out), *case)
    rows_of(b, off_out).fill_(3.0)
    assert b.eq(3.0).all()  # nothing between the rows was written
    call(qmm, rows_of(a, off_in), *case[1:], out=rows_of(a, off_in))  # in place
    check(rows_of(a.cpu(), off_in), *case)


def test_parts_may_be_left_out(qmm):
    x, h, prompt, rep, freq, pres, bias, allowed = make(np.random.default_rng(8), 4, 700, 90, 20)
    one, zero, none = np.ones(4, np.float32), np.zeros(4, np.float32), [[] for _ in range(4)]
    y = call(qmm, x, h, prompt, rep, freq, pres, bias, None)
    check(y, x, h, prompt, rep, freq, pres, bias, None)
    y = call(qmm, x, h, prompt, rep, freq, pres, bias, allowed, repetition=None)
    check(y, x, h, prompt, one, freq, pres, bias, allowed)
    y = call(qmm, x, h, prompt, rep, freq, pres, bias, allowed, frequency=None, presence=None, prompt_len=None)
    check(y, x, h, prompt * 0, rep, zero, zero, bias, allowed)
    y = call(qmm, x, h, prompt, rep, freq, pres, bias, allowed, bias_ids=None, bias_values=None, bias_start=None)
    check(y, x, h, prompt, rep, freq, pres, none, allowed)
    y = call(qmm, x, h, prompt, rep, freq, pres, bias, allowed, history=None, hist_start=None)
    check(y, x, [a[:0] for a in h], prompt, rep, freq, pres, bias, allowed)
    xd = torch.from_numpy(x).cuda()
    out = torch.empty_like(xd)
    qmm.qmm_logits_adjust(xd, out)
    assert torch.equal(out, xd)


def test_repeated_entries_and_hot_tokens(qmm):
    """Thousands of the same id (counts past 16 bits) and one id biased many
    times: the sums keep their order, 1e8 absorbs what comes right after it."""
    vocab = 5000
    x = np.zeros((1, vocab), np.float32)
    h = [np.concatenate([np.full(70000, 4097), np.full(3, 7)])]
    bias = [[(11, 1e8), (11, 1.0), (11, -1e8), (12, 2.0), (11, 0.5)] * 40]
    zero = np.zeros(1, np.float32)
    y = call(qmm, x, h, np.array([0]), zero + 1, zero + 0.5, zero + 2, bias, None).cpu().numpy()[0]
    assert y[4097] == -(35000 + 2) and y[7] == -3.5
    s = np.float32(0)
    for t, v in bias[0]:
        if t == 11:
            s = np.float32(s + np.float32(v))
    assert y[11] == s and y[12] == 80.0


def test_rows_without_allowed_tokens_and_odd_logits(qmm):
    x = np.array([[1.0, -np.inf, np.inf, np.nan, 2.0]] * 2, np.float32)
    allowed = np.array([[False] * 5, [True, True, True, True, False]])
    none = [np.zeros(0, np.int64)] * 2
    one, zero = np.ones(2, np.float32), np.zeros(2, np.float32)
    y = call(qmm, x, none, np.zeros(2), one, zero, zero, [[], []], allowed).cpu().numpy()
    assert np.isneginf(y[0]).all()  # a masked NaN does not come through
    assert y[1, 0] == 1 and np.isneginf(y[1, 1]) and y[1, 2] == np.inf and np.isnan(y[1, 3]) and np.isneginf(y[1, 4])


def test_starts_outside_the_lists_are_recorded(qmm):
    x = torch.zeros(2, 100).cuda()
    out = torch.empty_like(x)
    h = torch.tensor([5, 6], dtype=torch.int32).cuda()
    for start in ([0, 1, 3], [-1, 1, 2], [0, 1 << 30, 2]):
        s = torch.tensor(start, dtype=torch.int32).cuda()
        qmm.qmm_logits_adjust(x, out, history=h, hist_start=s, presence=torch.ones(2).cuda())
        assert qmm.qmm_get_device_error() == qmm.QMM_ERR_INDEX
    with pytest.raises(ValueError):
        qmm.qmm_logits_adjust(x, out[:, :99])
    with pytest.raises(ValueError):
        qmm.qmm_logits_adjust(x.half(), out)
    with pytest.raises(ValueError):
        qmm.qmm_logits_adjust(x, out, presence=torch.ones(3).cuda())
    with pytest.raises(qmm.QmmError):
        qmm.qmm_logits_adjust(x, out, history=h)


def test_another_stream_and_a_graph(qmm):
    case = make(np.random.default_rng(3), 3, 2000, 50, 5)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        y = call(qmm, *case)
    side.synchronize()
    check(y, *case)
    xd = torch.from_numpy(case[0]).cuda()
    out, pres = torch.zeros_like(xd), torch.zeros(3).cuda()
    h, start = ragged(case[1], np.int32)
    qmm.qmm_logits_adjust(xd, out, history=h, hist_start=start, presence=pres)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qmm.qmm_logits_adjust(xd, out, history=h, hist_start=start, presence=pres)
    pres.fill_(2.0)
    g.replay()
    torch.cuda.synchronize()
    one, zero = np.ones(3, np.float32), np.zeros(3, np.float32)
    check(out, case[0], case[1], np.zeros(3), one, zero, zero + 2, [[], [], []], None)
