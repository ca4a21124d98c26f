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
