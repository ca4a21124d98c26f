"""A pair's row has the same bits whatever other pairs its expert has."""
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


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


@pytest.mark.parametrize("types", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)], ids=str)
@pytest.mark.parametrize("tokens,experts", [(20, 64), (20, 8), (20, 2), (300, 3)])
@pytest.mark.parametrize("k", [512, 288, 2048])
def test_a_row_does_not_depend_on_its_neighbours(qmm, types, tokens, experts, k):
    """Token 9's expert has 1 to 16 other tokens (300 tokens: to 280), before and behind it."""
    rng = np.random.default_rng(tokens + experts + k)
    n, mine = 48, 9
    bg, bu = dev(ref.blocks(rng, experts, n, k)), dev(ref.blocks(rng, experts, n, k))
    x = rng.standard_normal((tokens, k)).astype(np.float32)
    ones = torch.ones(tokens, 1, device="cuda")
    first = None
    for others in ([0, 1, 2, 3, 4, 5, 7, 8, 11, 16] if tokens == 20 else [0, 3, 31, 40, 100, 140, 200, 280]):
        ids = 1 + rng.integers(0, experts - 1, (tokens, 1))
        ids[rng.permutation(np.delete(np.arange(tokens), mine))[:others]] = 0
        ids[mine] = 0
        starts, pairs = ref.plan_of(ids, experts)
        h = torch.empty(tokens, n, dtype=types[1], device="cuda")
        qmm.qmm_experts_geglu_q4_0(bg, bu, dev(x, types[0]), h, dev(starts), dev(pairs), 1, n, k)
        y = torch.empty(tokens, n, dtype=types[1], device="cuda")
        qmm.qmm_experts_down_q4_0(bg, dev(x[pairs], types[0]), y, dev(ids.astype(np.int32)), ones, dev(starts), dev(pairs), n, k)
        row = h[int(np.flatnonzero(pairs == mine)[0])], y[mine]
        if first is None:
            first = row
        assert torch.equal(row[0], first[0]) and torch.equal(row[1], first[1]), others
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


@pytest.mark.parametrize("types", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)], ids=str)
@pytest.mark.parametrize("tokens,experts", [(12, 64), (12, 2), (200, 2)])
@pytest.mark.parametrize("k", [512, 288])
def test_rows_without_a_number(qmm, types, tokens, experts, k):
    """A NaN in a row makes all of its results NaN, an infinity of either sign none of them
    finite, also where its weights are 0; the other rows keep their bits."""
    rng = np.random.default_rng(tokens + experts + k)
    n = 48
    b = ref.blocks(rng, experts, n, k)
    row = b.reshape(experts, n, k // 32, 18)
    row[:, ::3, 0, 2:] = 0x88  # weights of 0
    row[:, 1, :, 2:] = 0x88    # and a whole row of them
    w = dev(b)
    ids = rng.integers(0, experts, (tokens, 1))
    starts, pairs = ref.plan_of(ids, experts)
    x = rng.standard_normal((tokens, k)).astype(np.float32)
    odd = x.copy()
    odd[1, 5], odd[4, 7], odd[6, 100], odd[7, k - 1] = np.nan, np.inf, -np.inf, np.nan
    ones = torch.ones(tokens, 1, device="cuda")
    got = []
    for rows in (x, odd):
        h = torch.empty(tokens, n, dtype=types[1], device="cuda")
        qmm.qmm_experts_geglu_q4_0(w, w, dev(rows, types[0]), h, dev(starts), dev(pairs), 1, n, k)
        y = torch.empty(tokens, n, dtype=types[1], device="cuda")
        qmm.qmm_experts_down_q4_0(w, dev(rows[pairs], types[0]), y, dev(ids.astype(np.int32)), ones, dev(starts), dev(pairs), n, k)
        by_token = torch.empty_like(h)
        by_token[torch.from_numpy(pairs).long().cuda()] = h
        got.append((by_token, y))
    for plain, rows in zip(*got):
        assert torch.isnan(rows[[1, 7]]).all() and not torch.isfinite(rows[[4, 6]]).any()
        keep = np.delete(np.arange(tokens), [1, 4, 6, 7])
        assert torch.equal(plain[keep], rows[keep])
    assert qmm.qmm_get_device_error() == qmm.QMM_OK
