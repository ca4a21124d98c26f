"""Prompts' attention in the form that takes 128 or 256 query rows at a time:
whole blocks, and blocks whose keys are split among several CTAs.  That form is
chosen where the page table allows long contexts and the requests bring enough
rows, so that the tables here are wide, with unused entries of -1."""
import numpy as np
import pytest

import test_gpu_attn as base

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
qmm = base.qmm


class Wide(base.Case):
    def __init__(self, qmm, lens, new, heads, kv_heads, dim, page, keys=1 << 20, **kw):
        super().__init__(qmm, lens, new, heads, kv_heads, dim, page, **kw)
        table = np.full((len(lens), max(self.table.shape[1], keys // page)), -1)
        table[:, :self.table.shape[1]] = self.table
        self.table = table
        self.dev["table"] = torch.from_numpy(table.astype(np.int32)).cuda()

    def upload(self, qmm):
        self.cache = qmm.KvCacheQ4_0(*(torch.from_numpy(a).cuda() for a in self.arrays))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("q_type", [F32, BF16])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 1), (True, 40), (True, 200), (False, 0)])
def test_prompts_and_masks(qmm, dim, q_type, causal, window):
    lens, new = [70, 20, 129, 33, 300, 0, 5, 64], [70, 25, 1, 0, 140, 3, 2, 64]
    c = Wide(qmm, lens, new, 16, 2, dim, 32, seed=window, q_type=q_type)
    c.check(c.call(qmm, BF16, causal=causal, window=window), causal=causal, window=window)
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64), (256, 1024)])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 150), (True, 2500), (False, 0)])
@pytest.mark.parametrize("lens,new", [([5000, 3, 1200], [40, 3, 100]), ([20001], [33]), ([4096, 4097], [64, 64]),
                                      ([513, 512, 511, 1025], [100, 30, 1, 200])])
def test_split_contexts(qmm, dim, page, causal, window, lens, new):
    """Few rows and long contexts: a block's keys go to several CTAs; shorter
    ones beside it stay whole."""
    c = Wide(qmm, lens, new, 16, 2, dim, page, seed=len(lens), q_type=BF16)
    got = c.call(qmm, BF16, causal=causal, window=window)
    c.check(got, causal=causal, window=window)
    again = c.call(qmm, BF16, causal=causal, window=window)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_many_blocks_with_one_long_context(qmm, dim):
    """More blocks than three quarters of the SMs: only the long context is split."""
    lens, new = [6000] + [130 + 7 * i for i in range(60)], [40] + [30] * 60
    c = Wide(qmm, lens, new, 32, 2, dim, 64, seed=dim, q_type=BF16)
    c.check(c.call(qmm, BF16))
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_whole_blocks_of_a_window(qmm, dim):
    """A window bounds a block's keys: nothing is split."""
    c = Wide(qmm, [900], [800], 32, 2, dim, 64, seed=dim, q_type=BF16)
    c.check(c.call(qmm, BF16, window=150), window=150)
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lens,new", [([500, 90], [90, 90]), ([3000, 700], [24, 24])])
def test_sharp_and_wide_scores(qmm, dim, lens, new):
    c = Wide(qmm, lens, new, 8, 1, dim, 16, seed=3, spread=12.0)
    c.check(c.call(qmm, BF16))
    c.scale = 0.0
    c.check(c.call(qmm, BF16))
    c.scale = -0.05
    c.check(c.call(qmm, BF16))


@pytest.mark.parametrize("k_size,v_size,q_size", [(1, 4000.0, 1), (1, 2.0 ** -14, 1), (2.0 ** -10, 1, 2.0 ** 12),
                                                  (2000.0, 1, 2.0 ** -14), (1, 1, 1e-30), (2.0 ** -16, 1, 1e7)])
def test_sizes_of_values(qmm, k_size, v_size, q_size):
    c = Wide(qmm, [130, 1100], [100, 100], 4, 1, 64, 16, seed=5, spread=q_size)
    for i, size in ((1, k_size), (3, v_size)):
        c.arrays[i] = (c.arrays[i].astype(np.float32) * size).astype(np.float16)
    c.upload(qmm)
    c.check(c.call(qmm, BF16))


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_value_scales_that_differ_between_the_parts(qmm, dim):
    c = Wide(qmm, [2048], [80], 8, 1, dim, 64, seed=11)
    for i, pg in enumerate(c.table[0, :32]):
        c.arrays[3][pg] = (c.arrays[3][pg].astype(np.float32) * 2.0 ** (12 - abs(24 - 1.5 * i))).astype(np.float16)
    c.upload(qmm)
    c.check(c.call(qmm, BF16))


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_blocks_of_very_different_scales(qmm, dim):
    c = Wide(qmm, [200, 1300], [70, 70], 4, 1, dim, 32, seed=dim + 70)
    step = np.float32(2.0) ** -(np.arange(dim // 32) * 12 // max(1, dim // 32 - 1))
    for i in (1, 3):
        c.arrays[i] = (c.arrays[i].astype(np.float32) * step).astype(np.float16)
    c.upload(qmm)
    c.q = (c.q / torch.from_numpy(np.repeat(step, 32))).float()
    c.check(c.call(qmm, BF16))


@pytest.mark.parametrize("lens", [[120, 150], [1200, 2500]])
def test_a_nan_in_a_seen_key_or_query_stays_in_its_rows(qmm, lens):
    new = 100
    c = Wide(qmm, lens, [new, new], 8, 2, 64, 16, seed=4)
    c.arrays[1][c.table[1, 0], 1, 3] = np.nan   # a key of head 1 of the second request
    c.q[0, 7, 7] = float("nan")                 # a query of head 7
    c.upload(qmm)
    out, _ = c.call(qmm, BF16)
    want = np.zeros(out.shape, bool)
    want[new:, 4:] = True
    want[0, 7] = True
    assert np.array_equal(torch.isnan(out).cpu().numpy(), want)


@pytest.mark.parametrize("q_off,out_off", [(0, 0), (1, 3), (4, 2)])
@pytest.mark.parametrize("q_type", [F32, BF16])
@pytest.mark.parametrize("long", [90, 1900])
def test_strided_rows(qmm, q_off, out_off, q_type, long):
    c = Wide(qmm, [long, 200], [66, 1], 8, 2, 64, 32, seed=6, q_type=q_type)
    c_rows, wide = c.q.shape[0], 8 * 64 + 9
    basis = torch.zeros(c_rows * wide + 16, dtype=q_type)
    torch.as_strided(basis, (c_rows, 8, 64), (wide, 64, 1), q_off).copy_(c.q)
    q = torch.as_strided(basis.cuda(), (c_rows, 8, 64), (wide, 64, 1), q_off)
    dst = torch.full((c_rows * wide + 16,), 5.0, dtype=BF16).cuda()
    _, lse = c.call(qmm, BF16, q=q, out=torch.as_strided(dst, (c_rows, 8, 64), (wide, 64, 1), out_off))
    dst = dst.cpu()
    out = torch.as_strided(dst, (c_rows, 8, 64), (wide, 64, 1), out_off)
    c.check((out, lse))
    out.fill_(5.0)
    assert dst.eq(5.0).all()  # nothing between the rows was written


def test_one_graph_for_other_lengths(qmm):
    big = Wide(qmm, [4000, 500, 300], [120, 120, 1], 8, 2, 128, 16, seed=8)
    small = Wide(qmm, [120, 2160, 0], [120, 1, 120], 8, 2, 128, 16, seed=8)
    q = big.q.cuda()
    out, lse = torch.empty(q.shape, dtype=BF16).cuda(), torch.empty(q.shape[:2]).cuda()
    args = dict(max_q=120, scale=big.scale, lse=lse, workspace=qmm.attn_workspace(big.cache, 8), **big.dev)
    qmm.qmm_attn_q4_0(big.cache, q, out, **args)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qmm.qmm_attn_q4_0(big.cache, q, out, **args)
    g.replay()
    torch.cuda.synchronize()
    big.check((out, lse))
    # other lengths of the same requests (the second shares the first one's pages)
    table = big.table.copy()
    table[1] = table[0]
    small.arrays, small.table, small.q = big.arrays, table, big.q[:int(small.q_start[-1])]
    big.dev["table"].copy_(torch.from_numpy(table.astype(np.int32)))
    big.dev["q_start"].copy_(small.dev["q_start"])
    big.dev["kv_len"].copy_(small.dev["kv_len"])
    g.replay()
    torch.cuda.synchronize()
    n = small.q.shape[0]
    small.check((out[:n], lse[:n]))
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


@pytest.mark.parametrize("first", [100, 1800])
def test_bad_indices_are_left_out_and_recorded(qmm, first):
    new = 100
    c = Wide(qmm, [first, 100], [new, new], 8, 2, 64, 16, seed=10, keys=1 << 19)
    good = c.call(qmm, BF16)
    assert qmm.qmm_get_device_error() == qmm.QMM_OK
    for page in (-1, c.cache.num_pages, 1 << 30):
        t = c.dev["table"].clone()
        t[0, 1] = page
        out = torch.empty_like(good[0])
        qmm.qmm_attn_q4_0(c.cache, c.q.cuda(), out, t, c.dev["q_start"], c.dev["kv_len"], new, c.scale)
        assert qmm.qmm_get_device_error() == qmm.QMM_ERR_INDEX
        assert torch.equal(out[new:], good[0][new:]) and torch.isfinite(out).all()
    # rows that several requests claim
    start = torch.tensor([0, 2 * new, new], dtype=torch.int32).cuda()
    out = torch.empty_like(good[0])
    qmm.qmm_attn_q4_0(c.cache, c.q.cuda(), out, c.dev["table"], start, c.dev["kv_len"], new, c.scale)
    assert qmm.qmm_get_device_error() == qmm.QMM_ERR_INDEX


def test_another_stream(qmm):
    c = Wide(qmm, [3000, 800], [50, 50], 8, 2, 256, 64, seed=9, q_type=BF16)
    side = torch.cuda.Stream()
    q = c.q.cuda()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = c.call(qmm, BF16, q=q)
    side.synchronize()
    c.check(got)
