"""Attention at the ends of its arguments, in both forms (tables of the
requests' own width, and wide ones, which select the form of many rows)."""
import numpy as np
import pytest

import serving_ref as ref
import test_gpu_attn as base
from test_gpu_attn_prompts import Wide

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
qmm = base.qmm
FORMS = [(base.Case, F32), (base.Case, BF16), (Wide, BF16)]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("starts", [[0, 1000, 0, 1000], [0, 1000, 0, 1000, 0, 1000, 0, 1000]])
def test_rows_claimed_twice_keep_to_their_arrays(qmm, dim, starts):
    """Each way back claims all rows again, which makes more blocks and parts
    than total_q lets the launch expect: nothing outside the rows is written
    and the error is recorded."""
    rows, batch = 1000, len(starts) - 1
    lens = [rows if i % 2 == 0 else 0 for i in range(batch - 1)] + [32000]
    c = base.Case(qmm, lens, [rows] + [0] * (batch - 1), 8, 2, dim, 64, seed=dim, q_type=BF16)
    c.dev["q_start"] = torch.tensor(starts, dtype=torch.int32).cuda()
    guard, q = 64, c.q.cuda()
    out = torch.full((rows + 2 * guard, 8, dim), 7.0, dtype=BF16).cuda()
    lse = torch.full((rows + 2 * guard, 8), 7.0).cuda()
    ws = qmm.attn_workspace(c.cache, 8)
    space = torch.full((ws.numel() + 512,), 255, dtype=torch.uint8).cuda()  # stale: no number, and counts of -1
    for fill in (255, 1):
        space.fill_(fill)
        qmm.qmm_attn_q4_0(c.cache, q, out[guard:-guard], max_q=rows, scale=c.scale, lse=lse[guard:-guard],
                          workspace=space[256:-256], **c.dev)
        assert qmm.qmm_get_device_error() == qmm.QMM_ERR_INDEX
        for t in (out, lse):
            assert t[:guard].eq(7.0).all() and t[-guard:].eq(7.0).all()
        assert space[:256].eq(fill).all() and space[-256:].eq(fill).all()


@pytest.mark.parametrize("given", ["object", "handle"])
def test_a_workspace_of_its_own_belongs_to_its_stream(qmm, given):
    """Without a workspace, on a stream that is not the current one: the memory
    that the call takes must not serve the current stream while it runs."""
    c = base.Case(qmm, [9000, 800], [1, 1], 8, 2, 256, 64, seed=9)
    q, size = c.q.cuda(), qmm.attn_workspace(c.cache, 8).numel()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.empty(size, dtype=torch.uint8, device="cuda")  # the pools of both streams have room
    torch.cuda.synchronize()
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2]).cuda()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # some ms: the call waits behind it
    qmm.qmm_attn_q4_0(c.cache, q, out, max_q=1, scale=c.scale, lse=lse,
                      stream=side if given == "object" else side.cuda_stream, **c.dev)
    assert torch.cuda.current_stream() != side
    other = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
    side.synchronize()
    torch.cuda.synchronize()
    assert all(t.eq(255).all() for t in other)
    c.check((out, lse))
    # the default stream by its handle
    qmm.qmm_attn_q4_0(c.cache, q, out, max_q=1, scale=c.scale, lse=lse, stream=0, **c.dev)
    torch.cuda.synchronize()
    c.check((out, lse))


@pytest.mark.parametrize("lens,new", [([4000, 300], [1, 1]), ([3000, 900], [200, 100])])
def test_the_largest_window_is_no_window(qmm, lens, new):
    """The same form is taken, so the same bits come out."""
    c = base.Case(qmm, lens, new, 8, 2, 128, 64, seed=21, q_type=BF16)
    want = c.call(qmm, BF16)
    for window in (2 ** 31 - 1, 2 ** 31 - 64):
        got = c.call(qmm, BF16, window=window)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("form,out_type", FORMS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 60])
@pytest.mark.parametrize("long", [130, 1900])
def test_a_nan_in_a_seen_value_stays_in_its_dimensions(qmm, form, out_type, dim, window, long):
    """Neither lse nor the other blocks' outputs depend on it, nor do rows that
    do not see the key or read another key head."""
    new, page, block, key = 100, 16, 1, long - 40
    c = form(qmm, [long, 120], [new, new], 8, 2, dim, page, seed=dim, q_type=BF16)
    clean = [a.copy() for a in c.arrays]
    c.arrays[3][c.table[0, key // page], 1, key % page, block] = np.nan
    c.cache = qmm.KvCacheQ4_0(*(torch.from_numpy(a).cuda() for a in c.arrays))
    out, lse = c.call(qmm, out_type, window=window)
    pos = np.arange(long - new, long)
    rows = np.flatnonzero((pos >= key) & (pos < key + window if window else True))
    want = np.zeros(out.shape, bool)
    want[rows[0]:rows[-1] + 1, 4:, 32 * block:32 * block + 32] = True
    out = out.float().cpu()
    assert np.array_equal(torch.isnan(out).numpy(), want)
    # the rest is as without it
    c.arrays = clean
    truth = ref.attention(c.q.double().numpy(), *clean, c.table, c.q_start, c.lens, c.scale, True, window)
    lim_o, lim_l = ref.attention_limits(*truth, bf16=out_type == BF16)
    assert (np.abs(out.numpy() - truth[0]) <= lim_o)[~want].all()
    assert (np.abs(lse.cpu().numpy() - truth[1]) <= lim_l).all()


@pytest.mark.parametrize("dim,spread", [(64, 4.0), (128, 10.0), (256, 3.0), (256, 30.0)])
@pytest.mark.parametrize("lens,new", [([700, 300], [300, 300]), ([4000, 1500], [70, 90])])
def test_sharp_scores_and_zero_dimensions(qmm, dim, spread, lens, new):
    """Weights over a range that binary16 does not have, and a block of values
    that is 0 for every key, as where head dimensions are padded."""
    c = Wide(qmm, lens, new, 16, 2, dim, 64, seed=dim, q_type=BF16, spread=spread)
    c.arrays[3][..., -1] = 0
    c.upload(qmm)
    first = c.call(qmm, BF16)
    out, _ = c.check(first)
    assert (out[..., -32:] == 0).all()
    for _ in range(3):
        again = c.call(qmm, BF16)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


@pytest.mark.parametrize("dim", [128, 256])
@pytest.mark.parametrize("zero_block", [False, True])
def test_sharp_scores_take_a_few_passes_at_most(qmm, dim, zero_block):
    """Trained attention is sharp, and head dimensions are padded with zeros:
    neither may cost more than four passes over the keys, with room for the
    clock."""
    c = Wide(qmm, [4096], [1024], 16, 2, dim, 64, seed=dim, q_type=BF16)
    if zero_block:
        c.arrays[3][..., -1] = 0
        c.upload(qmm)
    ws, time = qmm.attn_workspace(c.cache, 16), []
    for spread in (0.1, 1.0, 4.0, 30.0):
        q = (c.q.float() * spread).to(BF16).cuda()
        out = torch.empty_like(q)
        call = lambda: qmm.qmm_attn_q4_0(c.cache, q, out, max_q=1024, scale=c.scale, workspace=ws, **c.dev)  # noqa: E731
        for _ in range(2):
            call()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(5):
            call()
        b.record()
        b.synchronize()
        time.append(a.elapsed_time(b) / 5)
    assert max(time) <= 6 * time[0], time


@pytest.mark.parametrize("dim", [128, 256])
@pytest.mark.parametrize("codes", [False, True])
def test_dimensions_without_values_take_no_passes(qmm, dim, codes):
    """Padded head dimensions, half a block of them: by scales of 0 or by codes
    of 0.  What cannot be other than 0 sends nothing over the keys again."""
    c = Wide(qmm, [4096], [1024], 16, 2, dim, 64, seed=dim, q_type=BF16)
    ws, q, out = qmm.attn_workspace(c.cache, 16), c.q.cuda(), torch.empty(c.q.shape, dtype=BF16).cuda()

    def time():
        call = lambda: qmm.qmm_attn_q4_0(c.cache, q, out, max_q=1024, scale=c.scale, workspace=ws, **c.dev)  # noqa: E731
        for _ in range(2):
            call()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(10):
            call()
        b.record()
        b.synchronize()
        return a.elapsed_time(b) / 10

    full = time()
    if codes:
        low = c.arrays[2][..., -16:]
        low[...] = (low & 15) | 0x80  # the last 16 dimensions
    else:
        c.arrays[3][..., -1] = 0
    c.upload(qmm)
    padded = time()
    assert (out[..., -16:] == 0).all() and not (out[..., -32:] == 0).all() == codes
    assert padded <= 1.25 * full, (padded, full)


@pytest.mark.parametrize("form,out_type", FORMS)
@pytest.mark.parametrize("long", [130, 1900])
def test_rows_beyond_max_q_are_left_out(qmm, form, out_type, long):
    c = form(qmm, [long, 120], [100, 50], 16, 2, 128, 16, seed=5, q_type=BF16)
    c.check(c.call(qmm, out_type))
    assert qmm.qmm_get_device_error() == qmm.QMM_OK
    want = ref.attention(c.q.double().numpy(), *c.arrays, c.table, c.q_start, c.lens, c.scale, True, 0)
    limit, limit_lse = ref.attention_limits(*want, bf16=out_type == BF16)
    out, lse = c.call(qmm, out_type, max_q=60)
    assert qmm.qmm_get_device_error() == qmm.QMM_ERR_INDEX
    out, lse = out.float().cpu().numpy(), lse.cpu().numpy()
    kept = np.r_[0:60, 100:150]  # of the first request its first 60 tokens, where they stand
    assert (out[60:100] == 7.0).all() and (lse[60:100] == 7.0).all()
    assert (np.abs(out - want[0]) <= limit)[kept].all() and (np.abs(lse - want[1]) <= limit_lse)[kept].all()


@pytest.mark.parametrize("form,out_type", FORMS)
@pytest.mark.parametrize("long", [130, 1900])
def test_rows_before_the_first_leave_the_others_in_place(qmm, form, out_type, long):
    c = form(qmm, [long, 120], [100, 50], 16, 2, 128, 16, seed=6, q_type=BF16)
    want = ref.attention(c.q.double().numpy(), *c.arrays, c.table, c.q_start, c.lens, c.scale, True, 0)
    limit, limit_lse = ref.attention_limits(*want, bf16=out_type == BF16)
    c.q = c.q[3:]
    c.dev["q_start"] -= 3
    out, lse = c.call(qmm, out_type)
    assert qmm.qmm_get_device_error() == qmm.QMM_ERR_INDEX
    assert (np.abs(out.float().cpu().numpy() - want[0][3:]) <= limit[3:]).all()
    assert (np.abs(lse.cpu().numpy() - want[1][3:]) <= limit_lse[3:]).all()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("out_type", [F32, BF16])
@pytest.mark.parametrize("span", [10, 16, 24])
@pytest.mark.parametrize("new", [1, 30])
def test_small_blocks_of_values_keep_their_bits(qmm, dim, out_type, span, new):
    """Value scales that fall by 2^span from the first block of a head to the
    last: each block's outputs are right by their own size."""
    for seed in range(3):
        c = base.Case(qmm, [200, 1300], [new, new], 8, 1, dim, 32, seed=span + 100 * seed, q_type=BF16)
        s = c.arrays[3].astype(np.float32)
        step = np.float32(2.0) ** -(np.arange(dim // 32) * span // (dim // 32 - 1))
        c.arrays[3] = (s / np.nanmax(s) * 16 * step).astype(np.float16)
        c.cache = qmm.KvCacheQ4_0(*(torch.from_numpy(a).cuda() for a in c.arrays))
        c.check(c.call(qmm, out_type))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("spread", [1.0, 12.0])
@pytest.mark.parametrize("new,window", [(1, 0), (3, 0), (30, 40)])
def test_bf16_queries_enter_the_streaming_form_exactly(qmm, dim, spread, new, window):
    """Where q is bf16 and the codes are used as they are, only sums and weights
    round.  A block's product of integers 0..15 with q, less 8 times q's sum,
    is formed in sums that keep 18 bits of their largest term; with B = scale *
    max_j sum_d (n + 8) d |q| a score is off by less than B * 2^-15 (a block
    takes two sums of 16 terms).  p, p d and the output round once to 11, 11
    and 8 bits:
        |out - ref| <= S * (2 * B * 2^-15 + 2^-10) + 2^-8 * |ref| + 1e-30
        |lse - ref| <= B * 2^-15 + 2^-18 * (1 + |lse|)
    which, at scores of some hundred, is far below the bound for q and k of 11
    bits."""
    c = base.Case(qmm, [300, 90], [new, new], 8, 2, dim, 16, seed=dim + new, q_type=BF16, spread=spread)
    out, lse = c.call(qmm, BF16, window=window)
    q = c.q.double().numpy()
    want, want_lse, _, share = ref.attention(q, *c.arrays, c.table, c.q_start, c.lens, c.scale, True, window)
    codes = [a.copy() for a in c.arrays[:2]]
    n = np.concatenate([codes[0].reshape(*codes[0].shape[:-1], -1, 16) & 15,
                        codes[0].reshape(*codes[0].shape[:-1], -1, 16) >> 4], -1).astype(np.float64) + 8
    size = (n * np.abs(codes[1].astype(np.float64))[..., None]).reshape(*codes[0].shape[:-1], -1)
    big = np.zeros(want_lse.shape)
    for b, length in enumerate(c.lens):
        rows = slice(int(c.q_start[b]), int(c.q_start[b + 1]))
        ids = c.table[b, :-(-length // 16)]
        for h in range(2):
            k = size[ids, h].reshape(-1, dim)[:length]
            big[rows, 4 * h:4 * h + 4] = (np.abs(q[rows, 4 * h:4 * h + 4]) @ k.T).max(-1) * c.scale
    limit = share * (2 * big[..., None] * 2.0 ** -15 + 2.0 ** -10) + 2.0 ** -8 * np.abs(want) + 1e-30
    assert (np.abs(out.double().cpu().numpy() - want) <= limit).all()
    assert (np.abs(lse.cpu().numpy() - want_lse) <= big * 2.0 ** -15 + 2.0 ** -18 * (1 + np.abs(want_lse))).all()


@pytest.mark.parametrize("form,out_type", FORMS)
@pytest.mark.parametrize("first", [100, 1800])
def test_every_negative_page_is_a_missing_one(qmm, form, out_type, first):
    """-2 as well as -1: the keys are left out and recorded."""
    c = form(qmm, [first, 100], [100, 100], 8, 2, 64, 16, seed=10)
    outs = []
    for page in (-1, -2, -3, -(2 ** 31)):
        t = c.dev["table"].clone()
        t[0, 1] = page
        out, lse = torch.empty(c.q.shape, dtype=out_type).cuda(), torch.empty(c.q.shape[:2]).cuda()
        qmm.qmm_attn_q4_0(c.cache, c.q.cuda(), out, t, c.dev["q_start"], c.dev["kv_len"], 100, c.scale, lse=lse)
        assert qmm.qmm_get_device_error() == qmm.QMM_ERR_INDEX, page
        outs.append((out, lse))
    for out, lse in outs[1:]:
        assert torch.equal(out, outs[0][0]) and torch.equal(lse, outs[0][1])
