"""Plan, cache and logits at the ends of their arguments, and requests of the
generation loop that stop, go on and end."""
import numpy as np
import pytest

import serving_ref as ref
import test_gpu_kv as kv
import test_gpu_logits as lg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
qmm = kv.qmm


def test_plan_counts_only_tokens_that_have_a_row(qmm):
    """Too little capacity: q_start and kv_len agree, so that the rows that are
    there stand at their positions."""
    cached, added = np.array([16, 5, 40, 7]), np.array([20, 40, 9, 0])
    table = np.full((4, 9), 3)
    for cap, kept in ((69, [20, 40, 9, 0]), (68, [20, 40, 8, 0]), (60, [20, 40, 0, 0]), (30, [20, 10, 0, 0]),
                      (20, [20, 0, 0, 0]), (3, [3, 0, 0, 0]), (0, [0, 0, 0, 0])):
        got = kv.run_plan(qmm, cached, added, np.arange(20), table, 16, cap)
        assert qmm.qmm_get_device_error() == (qmm.QMM_OK if cap == 69 else qmm.QMM_ERR_INDEX)
        assert got[1].tolist() == [0, *np.cumsum(kept)]
        assert got[2].tolist() == (cached + kept).tolist()


def test_a_slot_given_twice_spoils_no_other(qmm):
    """What stands in it is not defined; its neighbours are as they were."""
    cache = qmm.kv_cache_q4_0(2, 16, 2, 128)
    x = torch.randn(300, 2, 128).cuda()
    qmm.qmm_kv_append_q4_0(cache, x[:32], x[:32], torch.arange(32).cuda())
    before = [a.copy() for a in kv.cache_arrays(cache)]
    qmm.qmm_kv_append_q4_0(cache, x, x, torch.full((300,), 21).cuda())
    for a, b in zip(before, kv.cache_arrays(cache)):
        a[1, :, 5], b[1, :, 5] = 0, 0
        assert np.array_equal(a, b)
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


@pytest.mark.parametrize("vocab,extra,mask", [(262144, 0, False), (50001, 9000, True), (3000, 20000, True)])
def test_long_bias_lists(qmm, vocab, extra, mask):
    """A bias for every token, and ids that come several times: sums in list
    order, in a time that grows with the list and not with its square."""
    rng = np.random.default_rng(vocab)
    x, h, prompt, rep, freq, pres, _, allowed = lg.make(rng, 2, vocab, 500, 0)
    def entries():
        ids = np.concatenate([rng.permutation(vocab), rng.integers(-2, vocab + 2, extra)])
        rng.shuffle(ids)
        return [(int(t), float(np.float32(v))) for t, v in zip(ids, rng.standard_normal(len(ids)))]
    bias = [entries(), entries()[:700]]
    case = (x, h, prompt, rep, freq, pres, bias, allowed if mask else None)
    y = lg.call(qmm, *case)
    lg.check(y, *case)
    z = torch.from_numpy(x).cuda()
    lg.call(qmm, z, *case[1:], out=z)  # in place
    assert torch.equal(y, z)
    f = lambda a, t: torch.from_numpy(np.asarray(a, t)).cuda()  # noqa: E731
    flat = [e for b in bias for e in b]
    kw = dict(bias_ids=f([t for t, _ in flat], np.int32), bias_values=f([v for _, v in flat], np.float32),
              bias_start=f([0, len(bias[0]), len(flat)], np.int32))
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    qmm.qmm_logits_adjust(z, z, **kw)
    b.record()
    b.synchronize()
    assert a.elapsed_time(b) < 10.0


def test_long_bias_lists_keep_the_order(qmm):
    """1e8 absorbs what comes right after it, beyond the entries kept aside too."""
    n = 3000
    rng = np.random.default_rng(1)
    ids = rng.integers(0, 40, n)
    vals = rng.choice(np.array([1e8, 1.0, -1e8, 0.5], np.float32), n)
    zero = np.zeros(1, np.float32)
    x = rng.standard_normal((1, 50)).astype(np.float32)
    y = lg.call(qmm, x, [np.zeros(0, np.int64)], np.array([0]), zero + 1, zero, zero,
                [[(int(t), float(v)) for t, v in zip(ids, vals)]], None).cpu().numpy()[0]
    s = np.zeros(50, np.float32)
    for t, v in zip(ids, vals):
        s[t] = np.float32(s[t] + v)
    assert np.array_equal(y, x[0] + s)


@pytest.fixture(scope="module")
def gen(qmm):
    from block_quantized_matmul_gguf_gb300 import generate
    return generate


def small_layer(gen):
    return gen.Layer(hidden=256, heads=4, kv_heads=2, head_dim=64, vocab=512, seed=3)


def test_a_request_without_new_tokens_answers_for_itself(gen):
    layer = small_layer(gen)
    g = gen.Generator(layer, 3)
    first = g.step([[1, 2, 3], [4] * 40, [9, 8]])
    second = g.step([[first[0]], [], [first[2]]])
    assert second[1] == first[1]  # its cache and its history are as they were
    assert g.kv_len.tolist() == [4, 40, 3]
    assert g.step([[], [], []]) == second
    assert g.kv_len.tolist() == [4, 40, 3]
    # beside others or alone, it goes on as if nothing had been between
    lone = gen.Generator(layer, 3)
    lone.step([[1, 2, 3], [4] * 40, [9, 8]])
    lone.step([[first[0]], [], [first[2]]])
    assert g.step([[], [first[1]], []])[1] == lone.step([[], [first[1]], []])[1]


def test_a_request_longer_than_its_table_row_is_refused(gen, qmm):
    g = gen.Generator(small_layer(gen), 2, max_pages=2)
    g.step([[1] * 30, [2]])
    with pytest.raises(RuntimeError):
        g.step([[1] * 3, [2]])
    assert g.kv_len.tolist() == [30, 1]
    g.step([[1] * 2, [2]])
    assert g.kv_len.tolist() == [32, 2] and qmm.qmm_get_device_error() == qmm.QMM_OK


def test_a_second_run_counts_its_own_tokens(gen):
    """What an earlier run brought is prompt to the next one."""
    layer = small_layer(gen)
    g = gen.Generator(layer, 1)
    made = g.run([[1, 2, 3]], 4)[0]
    before = list(g.history[0])
    assert before == [1, 2, 3] + made[:3]
    g.run([[5, 6]], 1)
    assert g.prompt_len.tolist() == [len(before) + 2]
