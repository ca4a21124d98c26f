"""Attention over the paged Q4_0 cache on the GPU against a plain 64-bit
reference (serving_ref.attention), within the bounds derived there."""
import numpy as np
import pytest

import serving_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def qmm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_quantized_matmul_gguf_gb300 import build, qmm as q
    build.build_library()
    q.load()
    q.qmm_get_device_error()
    return q


class Case:
    """A filled cache whose unused slots and pages hold NaN scales."""

    def __init__(self, qmm, lens, new, heads, kv_heads, dim, page, seed=0, q_type=F32, spread=1.0, extra_pages=2):
        rng = np.random.default_rng(seed)
        self.lens, self.new, self.dim, self.heads = list(lens), list(new), dim, heads
        need = [-(-n // page) for n in lens]
        pages = sum(need) + extra_pages
        ids = rng.permutation(pages)
        width = max(1, max(need) + 1)
        self.table = np.full((len(lens), width), -1)
        at = 0
        shape = (pages, kv_heads, page)
        self.arrays = []
        for _ in range(2):
            c = rng.integers(0, 256, (*shape, dim // 2), dtype=np.uint8)
            s = np.full((*shape, dim // 32), np.nan, np.float16)
            self.arrays += [c, s]
        for b, n in enumerate(lens):
            mine = ids[at:at + need[b]]
            at += need[b]
            self.table[b, :need[b]] = mine
            for i, pg in enumerate(mine):
                live = min(page, n - i * page)
                for half in range(2):
                    c, s = ref.quantize(rng.standard_normal((kv_heads, live, dim)) *
                                        np.exp(0.5 * rng.standard_normal((kv_heads, live, 1))))
                    self.arrays[2 * half][pg, :, :live] = c
                    self.arrays[2 * half + 1][pg, :, :live] = s
        self.q_start = np.concatenate([[0], np.cumsum(new)])
        rows = int(self.q_start[-1])
        self.q = (torch.from_numpy(rng.standard_normal((rows, heads, dim)).astype(np.float32)) * spread).to(q_type)
        self.cache = qmm.KvCacheQ4_0(*(torch.from_numpy(a).cuda() for a in self.arrays))
        self.scale = dim ** -0.5
        i32 = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()  # noqa: E731
        self.dev = dict(table=i32(self.table), q_start=i32(self.q_start), kv_len=i32(self.lens))

    def call(self, qmm, out_type, causal=True, window=0, max_q=None, q=None, out=None, **kw):
        q = self.q.cuda() if q is None else q
        out = torch.full(self.q.shape, 7.0, dtype=out_type).cuda() if out is None else out
        lse = torch.full(self.q.shape[:2], 7.0).cuda()
        qmm.qmm_attn_q4_0(self.cache, q, out, max_q=max_q or max(1, max(self.new)), scale=self.scale,
                          causal=causal, window=window, lse=lse, **self.dev, **kw)
        return out, lse

    def check(self, got, causal=True, window=0):
        out, lse = got
        want = ref.attention(self.q.float().numpy().astype(np.float64), *self.arrays, self.table, self.q_start,
                             self.lens, self.scale, causal, window)
        lim_o, lim_l = ref.attention_limits(*want, bf16=out.dtype == BF16)
        o, z = out.float().cpu().numpy(), lse.cpu().numpy()
        empty = np.isneginf(want[1])
        assert np.array_equal(np.isneginf(z), empty)
        assert (o[empty] == 0).all()
        bad = ~(np.abs(o - want[0]) <= lim_o)
        assert not bad.any(), (np.argwhere(bad)[:4].tolist(), o[bad][:4], want[0][bad][:4], lim_o[bad][:4])
        assert (np.abs(z[~empty] - want[1][~empty]) <= lim_l[~empty]).all()
        return o, want[0]


TYPES = [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (2, 1), (4, 1), (8, 2), (6, 2), (5, 1), (16, 2), (24, 2), (3, 3)])
@pytest.mark.parametrize("out_type", [F32, BF16])
def test_head_layouts(qmm, dim, heads, kv_heads, out_type):
    c = Case(qmm, [37, 130, 1], [1, 1, 1], heads, kv_heads, dim, 16, seed=dim + heads)
    c.check(c.call(qmm, out_type))
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


@pytest.mark.parametrize("dim,page", [(64, 16), (64, 1024), (128, 32), (128, 64), (256, 16), (256, 128)])
@pytest.mark.parametrize("q_type,out_type", TYPES)
def test_lengths(qmm, dim, page, q_type, out_type):
    """Every kind of end: empty requests, one key, ends inside and at the
    edges of blocks, tiles and pages."""
    lens = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 300, 1025]
    c = Case(qmm, lens, [1] * len(lens), 8, 2, dim, page, seed=page, q_type=q_type)
    c.check(c.call(qmm, out_type))
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("q_type,out_type", TYPES)
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 1), (True, 40), (True, 200), (False, 0)])
def test_prompts_and_masks(qmm, dim, q_type, out_type, causal, window):
    """Ragged prompts with single tokens and none at all between them; the
    second request has fewer keys than tokens, so its first rows see none."""
    lens, new = [70, 20, 129, 33, 300, 0, 5, 64], [70, 25, 1, 0, 140, 3, 2, 64]
    c = Case(qmm, lens, new, 4, 2, dim, 32, seed=window, q_type=q_type)
    c.check(c.call(qmm, out_type, causal=causal, window=window), causal=causal, window=window)
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


@pytest.mark.parametrize("heads,kv_heads,dim,new,lens", [
    (8, 2, 256, [257, 3], [700, 3]), (8, 8, 64, [300], [300]), (16, 1, 128, [130], [1000]),
    (10, 2, 128, [129, 64, 1], [129, 600, 900]), (4, 1, 64, [513], [515]), (2, 1, 256, [1000], [1000]),
])
@pytest.mark.parametrize("out_type", [F32, BF16])
@pytest.mark.parametrize("window", [0, 150])
def test_long_prompts(qmm, heads, kv_heads, dim, new, lens, out_type, window):
    c = Case(qmm, lens, new, heads, kv_heads, dim, 64, seed=heads, q_type=F32)
    c.check(c.call(qmm, out_type, window=window), window=window)
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


@pytest.mark.parametrize("dim,heads,kv_heads", [(256, 8, 2), (128, 16, 4), (64, 8, 1)])
def test_prompts_give_the_same_bits_every_time(qmm, dim, heads, kv_heads):
    c = Case(qmm, [1500, 700, 333], [900, 700, 64], heads, kv_heads, dim, 32, seed=dim, q_type=BF16)
    first = c.call(qmm, BF16)
    for _ in range(30):
        again = c.call(qmm, BF16)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


@pytest.mark.parametrize("dim,page,n,out_type", [(256, 16, 20011, F32), (128, 64, 50000, BF16), (64, 128, 30001, F32)])
def test_long_contexts(qmm, dim, page, n, out_type):
    """One request over the whole GPU, beside short ones."""
    lens = [n, 3, 700]
    c = Case(qmm, lens, [1, 1, 2], 8, 2, dim, page, seed=n)
    a = c.call(qmm, out_type)
    o, want = c.check(a)
    rel = np.linalg.norm(o - want) / np.linalg.norm(want)
    assert rel <= (4e-3 if out_type == BF16 else 1e-5)  # bf16: 2^-8
    b = c.call(qmm, out_type)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])  # the same bits every time
    c.check(c.call(qmm, out_type, window=1500), window=1500)


@pytest.mark.parametrize("out_type", [F32, BF16])
@pytest.mark.parametrize("new", [1, 3, 90])
def test_sharp_and_wide_scores(qmm, out_type, new):
    """Scores of some hundred: one key takes the whole weight; and equal ones."""
    c = Case(qmm, [500, 90], [new, new], 8, 2, 128, 16, seed=3, spread=12.0)
    c.check(c.call(qmm, out_type))
    c.scale = 0.0
    c.check(c.call(qmm, out_type))
    c.scale = -0.05
    c.check(c.call(qmm, out_type))


@pytest.mark.parametrize("new", [1, 4, 100])
@pytest.mark.parametrize("k_size,v_size,q_size", [(1, 4000.0, 1), (1, 2.0 ** -14, 1), (2.0 ** -10, 1, 2.0 ** 12),
                                                  (2000.0, 1, 2.0 ** -14), (1, 1, 1e-30), (2.0 ** -16, 1, 1e7)])
def test_sizes_of_values(qmm, new, k_size, v_size, q_size):
    """Large and tiny scales of keys, values and queries, up to the ends of
    binary16: nothing overflows or loses its bits."""
    for out_type in (F32, BF16):
        c = Case(qmm, [130, 300], [new, new], 4, 1, 64, 16, seed=int(new), spread=q_size)
        for i, size in ((1, k_size), (3, v_size)):
            s = c.arrays[i].astype(np.float32) * size
            c.arrays[i] = s.astype(np.float16)
        c.cache = qmm.KvCacheQ4_0(*(torch.from_numpy(a).cuda() for a in c.arrays))
        c.check(c.call(qmm, out_type))


def test_mixed_sizes_within_a_request(qmm):
    """Value scales that grow by 2^24 along the context and fall again."""
    for out_type in (F32, BF16):
        for new in (1, 80):
            c = Case(qmm, [640], [new], 4, 1, 64, 64, seed=11)
            for i, pg in enumerate(c.table[0, :10]):
                c.arrays[3][pg] = (c.arrays[3][pg].astype(np.float32) * 2.0 ** (12 - abs(24 - 5 * i))).astype(np.float16)
            c.cache = qmm.KvCacheQ4_0(*(torch.from_numpy(a).cuda() for a in c.arrays))
            c.check(c.call(qmm, out_type))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 70])
def test_blocks_of_very_different_scales(qmm, dim, new):
    """Head dimensions whose scales differ by 2^12 within a key, with queries
    that make up for it: every block counts."""
    for out_type in (F32, BF16):
        c = Case(qmm, [200, 130], [new, new], 4, 1, dim, 32, seed=dim + new)
        step = np.float32(2.0) ** -(np.arange(dim // 32) * 12 // max(1, dim // 32 - 1))
        for i in (1, 3):
            c.arrays[i] = (c.arrays[i].astype(np.float32) * step).astype(np.float16)
        c.cache = qmm.KvCacheQ4_0(*(torch.from_numpy(a).cuda() for a in c.arrays))
        c.q = (c.q / torch.from_numpy(np.repeat(step, 32))).float()
        c.check(c.call(qmm, out_type))


def test_zero_scales_and_zero_queries(qmm):
    for new in (1, 70):
        c = Case(qmm, [100], [new], 4, 1, 128, 16, seed=2)
        c.arrays[1][c.table[0, 0]] = 0   # keys of zero
        c.arrays[3][:] = 0               # all values zero
        c.q[0] = 0
        c.cache = qmm.KvCacheQ4_0(*(torch.from_numpy(a).cuda() for a in c.arrays))
        for out_type in (F32, BF16):
            o, _ = c.check(c.call(qmm, out_type))
            assert (o == 0).all()


@pytest.mark.parametrize("new", [1, 100])
def test_a_nan_in_a_seen_key_or_query_stays_in_its_rows(qmm, new):
    c = Case(qmm, [120, 150], [new, new], 4, 2, 64, 16, seed=4)
    c.arrays[1][c.table[1, 0], 1, 3] = np.nan   # a key of head 1 of the second request
    c.q[0, 3, 7] = float("nan")                 # a query of head 3
    c.cache = qmm.KvCacheQ4_0(*(torch.from_numpy(a).cuda() for a in c.arrays))
    for out_type in (F32, BF16):
        out, _ = c.call(qmm, out_type)
        nan = torch.isnan(out).cpu().numpy()
        want = np.zeros(nan.shape, bool)
        want[new:, 2:] = True
        want[0, 3] = True
        assert np.array_equal(nan, want)


@pytest.mark.parametrize("q_off,out_off", [(0, 0), (1, 3), (4, 2)])
@pytest.mark.parametrize("new", [1, 66])
def test_strided_rows(qmm, q_off, out_off, new):
    for q_type, out_type in TYPES:
        c = Case(qmm, [90, 200], [new, 1], 4, 2, 64, 32, seed=6, q_type=q_type)
        rows, wide = c.q.shape[0], 4 * 64 + 9
        base = torch.zeros(rows * wide + 16, dtype=q_type)
        torch.as_strided(base, (rows, 4, 64), (wide, 64, 1), q_off).copy_(c.q)
        q = torch.as_strided(base.cuda(), (rows, 4, 64), (wide, 64, 1), q_off)
        dst = torch.full((rows * wide + 16,), 5.0, dtype=out_type).cuda()
        _, lse = c.call(qmm, out_type, q=q, out=torch.as_strided(dst, (rows, 4, 64), (wide, 64, 1), out_off))
        dst = dst.cpu()
        out = torch.as_strided(dst, (rows, 4, 64), (wide, 64, 1), out_off)
        c.check((out, lse))
        out.fill_(5.0)
        assert dst.eq(5.0).all()  # nothing between the rows was written


def test_rows_past_the_last_request_are_not_written(qmm):
    c = Case(qmm, [50, 60], [2, 40], 4, 2, 64, 16, seed=7)
    q = torch.cat([c.q.cuda(), torch.full((9, 4, 64), float("nan")).cuda()])
    for out_type in (F32, BF16):
        out = torch.full(q.shape, 3.0, dtype=out_type).cuda()
        lse = torch.full(q.shape[:2], 3.0).cuda()
        qmm.qmm_attn_q4_0(c.cache, q, out, max_q=40, scale=c.scale, lse=lse, **c.dev)
        out, lse = out.cpu(), lse.cpu()
        assert out[42:].eq(3.0).all() and lse[42:].eq(3.0).all()
        c.check((out[:42], lse[:42]))


@pytest.mark.parametrize("out_type", [F32, BF16])
@pytest.mark.parametrize("new", [1, 120])
def test_one_graph_for_other_lengths(qmm, out_type, new):
    big = Case(qmm, [400, 500, 300], [new, new, 1], 8, 2, 128, 16, seed=8)
    small = Case(qmm, [new, 40 + new, 0], [new, 1, new], 8, 2, 128, 16, seed=8)
    q = big.q.cuda()
    ws = qmm.attn_workspace(big.cache, 8)
    out, lse = torch.empty(q.shape, dtype=out_type).cuda(), torch.empty(q.shape[:2]).cuda()
    args = dict(max_q=max(big.new), scale=big.scale, lse=lse, workspace=ws, **big.dev)
    qmm.qmm_attn_q4_0(big.cache, q, out, **args)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qmm.qmm_attn_q4_0(big.cache, q, out, **args)
    g.replay()
    torch.cuda.synchronize()
    big.check((out, lse))
    # other lengths of the same requests: keys 0 .. n-1 of the same pages
    small.arrays, small.table, small.q = big.arrays, big.table, big.q[:int(small.q_start[-1])]
    big.dev["q_start"].copy_(small.dev["q_start"])
    big.dev["kv_len"].copy_(small.dev["kv_len"])
    g.replay()
    torch.cuda.synchronize()
    n = small.q.shape[0]
    small.check((out[:n], lse[:n]))
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


def test_another_stream(qmm):
    c = Case(qmm, [3000, 80], [1, 1], 8, 2, 256, 64, seed=9)
    side = torch.cuda.Stream()
    q = c.q.cuda()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = c.call(qmm, F32, q=q)
    side.synchronize()
    c.check(got)


@pytest.mark.parametrize("out_type", [F32, BF16])
@pytest.mark.parametrize("new", [1, 64])
def test_bad_indices_are_left_out_and_recorded(qmm, out_type, new):
    c = Case(qmm, [100, 100], [new, new], 4, 2, 64, 16, seed=10)
    good = c.call(qmm, out_type)
    assert qmm.qmm_get_device_error() == qmm.QMM_OK
    for page in (-1, c.cache.num_pages, 1 << 30):
        t = c.dev["table"].clone()
        t[0, 1] = page
        out = torch.empty_like(good[0])
        qmm.qmm_attn_q4_0(c.cache, c.q.cuda(), out, t, c.dev["q_start"], c.dev["kv_len"], new, c.scale)
        assert qmm.qmm_get_device_error() == qmm.QMM_ERR_INDEX
        assert torch.equal(out[new:], good[0][new:]) and torch.isfinite(out).all()
    # a length beyond the table
    long = torch.tensor([100, 1 << 30], dtype=torch.int32).cuda()
    out = torch.full_like(good[0], 2.0)
    qmm.qmm_attn_q4_0(c.cache, c.q.cuda(), out, c.dev["table"], c.dev["q_start"], long, new, c.scale)
    assert qmm.qmm_get_device_error() == qmm.QMM_ERR_INDEX
    assert torch.equal(out[:new], good[0][:new])
    # rows beyond q
    out = torch.full_like(good[0], 2.0)
    qmm.qmm_attn_q4_0(c.cache, c.q.cuda()[:new], out[:new], c.dev["table"], c.dev["q_start"], c.dev["kv_len"],
                      new, c.scale)
    assert qmm.qmm_get_device_error() == qmm.QMM_ERR_INDEX
    assert torch.equal(out[:new], good[0][:new]) and out[new:].eq(2.0).all()
    if new > 1:  # more tokens than max_q says
        qmm.qmm_attn_q4_0(c.cache, c.q.cuda(), out, c.dev["table"], c.dev["q_start"], c.dev["kv_len"], 1, c.scale)
        assert qmm.qmm_get_device_error() == qmm.QMM_ERR_INDEX


def test_cache_past_32_bit_offsets(qmm):
    """Pages whose codes lie beyond 4 GiB, for single tokens and prompts."""
    pages, page, heads, dim = 18000, 1024, 2, 256
    c = Case(qmm, [1500, 90], [1, 64], 8, heads, dim, page, seed=12)
    big = [torch.empty((pages, heads, page, w), dtype=t, device="cuda")
           for w, t in ((128, torch.uint8), (8, torch.float16)) * 2]
    place = {int(p): pages - 1 - 700 * i for i, p in enumerate(c.table[c.table >= 0])}
    for dst, src in zip(big, c.arrays):
        for p, to in place.items():
            dst[to] = torch.from_numpy(src[p]).cuda()
    table = torch.from_numpy(np.vectorize(lambda p: place.get(int(p), -1))(c.table).astype(np.int32)).cuda()
    c.cache = qmm.KvCacheQ4_0(*big)
    c.dev["table"] = table
    for out_type in (F32, BF16):
        c.check(c.call(qmm, out_type))
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


def test_python_refusals(qmm):
    c = Case(qmm, [20], [1], 4, 2, 64, 16)
    q, d = c.q.cuda(), c.dev
    out = torch.empty_like(q)
    for bad in (dict(q=q.half()), dict(out=out[:0]), dict(table=d["table"].long()), dict(kv_len=d["kv_len"].float()),
                dict(q_start=d["kv_len"]), dict(lse=torch.empty(3).cuda()), dict(q=c.q), dict(out=out[:, :2])):
        kw = dict(q=q, out=out, max_q=1, scale=0.1, **d)
        kw.update(bad)
        with pytest.raises(ValueError):
            qmm.qmm_attn_q4_0(c.cache, **kw)
    with pytest.raises(qmm.QmmError):
        qmm.qmm_attn_q4_0(c.cache, q, out, max_q=1, scale=0.1, causal=False, window=3, **d)
    with pytest.raises(qmm.QmmError):
        qmm.qmm_attn_q4_0(c.cache, q[:, :3], torch.empty(1, 3, 64).cuda(), max_q=1, scale=0.1, **d)
