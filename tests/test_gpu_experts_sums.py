"""The experts' products where what is added nearly cancels, so that a rounding on
the way shows beside the result's own."""
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


@pytest.mark.parametrize("types", [(BF16, BF16), (F32, BF16), (F32, F32)], ids=str)
@pytest.mark.parametrize("tokens,experts", [(3, 64), (3, 4), (90, 4)])
def test_projections_are_not_rounded_before_the_sum(qmm, types, tokens, experts):
    """Each token's two experts share all but one block in 32 of their weights, with
    weights 1 and -1: the sum is a quarter of either projection in size.  Rounding
    it leaves errors of random sign below 2^-8 |y|, whose root mean square is
    2^-8 / sqrt(3); the products may add 2^-11 |y| and the sum be off by less than 2^-8
    |y| in norm.  Projections rounded to bf16 would be off by some 2^-6.8 |y|."""
    rng = np.random.default_rng(tokens + experts)
    n, k, topk = 64, 1024, 2
    b = ref.blocks(rng, experts, n, k)
    b[1::2] = b[::2]
    row = b.reshape(experts, n, k // 32, 18)
    row[1::2, :, 7] = ref.blocks(rng, experts // 2, n, 32).reshape(-1, n, 18)
    first = 2 * rng.integers(0, experts // 2, tokens)
    ids = np.stack([first, first + 1], 1)
    starts, pairs = ref.plan_of(ids, experts)
    x = torch.from_numpy(rng.standard_normal((tokens, k)).astype(np.float32)).to(types[0])
    h = x[torch.from_numpy(pairs // topk).long()].cuda()
    weights = np.tile(np.float32([1, -1]), (tokens, 1))
    y = torch.empty(tokens, n, dtype=types[1], device="cuda")
    qmm.qmm_experts_down_q4_0(dev(b), h, y, dev(ids.astype(np.int32)), dev(weights), dev(starts), dev(pairs), n, k)
    w, _ = ref.matrix(b)
    want = np.einsum("tk,tnk->tn", x.double().numpy(), w[first] - w[first + 1])
    assert np.linalg.norm(y.double().cpu().numpy() - want) <= 2.0 ** -8 * np.linalg.norm(want)
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


TILES = [(3, 4), (90, 4)]  # tokens and experts that take the tile form


@pytest.mark.parametrize("k", [64, 256, 288, 1024])
@pytest.mark.parametrize("tokens,experts", TILES)
def test_weights_enter_whole(qmm, tokens, experts, k):
    """Each row of x holds v and -v where two blocks have one code c and scales that are
    neighbours in binary16.  v c (d - d') has every addend and sum within 24 bits, so
    that nothing but the result's rounding is left: half a step, 2^-8 |y|; the GELU
    adds 2^-11."""
    rng = np.random.default_rng(tokens + k)
    n = 48
    b = ref.blocks(rng, experts, n, k)
    row = b.reshape(experts, n, k // 32, 18)
    row[:, :, 1] = row[:, :, 0]
    d = row[:, :, 0, :2].copy().view(np.uint16) + np.uint16(1)  # the next scale
    row[:, :, 1, :2] = d.view(np.uint8)
    ids = rng.integers(0, experts, (tokens, 1))
    starts, pairs = ref.plan_of(ids, experts)
    at = rng.integers(0, 32, tokens)
    x = np.zeros((tokens, k), dtype=np.float32)
    v = torch.from_numpy(rng.uniform(50000, 100000, tokens).astype(np.float32)).bfloat16().float().numpy()
    x[np.arange(tokens), at], x[np.arange(tokens), 32 + at] = v, -v
    w, _ = ref.matrix(b)
    want = np.einsum("tk,tnk->tn", x.astype(np.float64), w[ids[:, 0]])[pairs]
    h = torch.empty(tokens, n, dtype=BF16, device="cuda")
    qmm.qmm_experts_geglu_q4_0(dev(b), dev(b), dev(x, BF16), h, dev(starts), dev(pairs), 1, n, k)
    z = ref.gelu(want) * want
    assert (np.abs(h.double().cpu().numpy() - z) <= (2.0 ** -8 + 2.0 ** -11) * np.abs(z) + 2.0 ** -11 * np.abs(want)).all()
    y = torch.empty(tokens, n, dtype=BF16, device="cuda")
    ones = torch.ones(tokens, 1, device="cuda")
    qmm.qmm_experts_down_q4_0(dev(b), dev(x[pairs], BF16), y, dev(ids.astype(np.int32)), ones, dev(starts), dev(pairs), n, k)
    assert (np.abs(y.double().cpu().numpy()[pairs] - want) <= 2.0 ** -8 * np.abs(want)).all()
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


@pytest.mark.parametrize("k", [256, 288])
@pytest.mark.parametrize("tokens,experts", TILES)
def test_scales_and_rows_of_any_range(qmm, tokens, experts, k):
    """Scales to the largest of binary16, whose weights that type cannot hold; and rows whose largest
    value, 1e30, meets weights of 0.  Bounds: those of exact products, and the result's rounding."""
    rng = np.random.default_rng(tokens + k)
    n, topk = 40, 2
    ids = np.argsort(rng.random((tokens, experts)), axis=1)[:, :topk]
    starts, pairs = ref.plan_of(ids, experts)
    weights = rng.random((tokens, topk)).astype(np.float32)
    h = torch.from_numpy(rng.standard_normal((tokens * topk, k)).astype(np.float32)).bfloat16()
    for lo, hi in ((8000, 65504), (0.001, 0.02), (6e-8, 1e-5)):
        b = ref.blocks(rng, experts, n, k, lo=lo, hi=hi)
        row = b.reshape(experts, n, k // 32, 18)
        row[:, :, 1, 2 + 5] = row[:, :, 1, 2 + 5] & 0xF0 | 8  # value 37 of each row of weights is 0
        clean = h.clone()
        clean[:, 37] = 0
        want, limit = ref.experts_down(clean.double().numpy(), b, ids, weights, starts, pairs, True, False)
        odd = clean.clone()
        odd[:, 37] = 1e30
        for rows in (clean, odd):
            y = torch.empty(tokens, n, dtype=BF16, device="cuda")
            qmm.qmm_experts_down_q4_0(dev(b), rows.cuda(), y, dev(ids.astype(np.int32)), dev(weights), dev(starts), dev(pairs), n, k)
            assert (np.abs(y.double().cpu().numpy() - want) <= limit + 2.0 ** -8 * (np.abs(want) + limit)).all()
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


@pytest.mark.parametrize("types", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)], ids=str)
@pytest.mark.parametrize("tokens,experts", [(3, 64), (7, 64), (1, 4), (90, 4)])
@pytest.mark.parametrize("k", [256, 288])
def test_inputs_and_codes_enter_whole(qmm, types, tokens, experts, k):
    """Rows that hold v in one place and -(v + 1) in another with the same weight w: y = -w.
    v has 13 bits (8 for bf16, where -(v + 1) is split over two places), so that the products
    of v and a code are exact and those with a scale off by 2^-24 of 2^13 w, twice: within
    2^-10 |w|, and the result's rounding of 2^-8 |w| or 2^-24."""
    rng = np.random.default_rng(tokens + experts + k)
    n = 48
    b = ref.blocks(rng, experts, n, k)
    row = b.reshape(experts, n, k // 32, 18)
    row[:, :, 1] = row[:, :, 0]
    row[:, :, 2] = row[:, :, 0]
    ids = rng.integers(0, experts, (tokens, 1))
    starts, pairs = ref.plan_of(ids, experts)
    at = rng.integers(0, 32, tokens)
    every = np.arange(tokens)
    x = np.zeros((tokens, k), dtype=np.float32)
    if types[0] is F32:
        v = rng.integers(1 << 12, (1 << 13) - 1, tokens).astype(np.float32)
        x[every, at], x[every, 32 + at] = v, -(v + 1)
    else:
        v = 32 * rng.integers(128, 256, tokens).astype(np.float32)
        x[every, at], x[every, 32 + at], x[every, 64 + at] = v, -v, -1
    w, _ = ref.matrix(b)
    want = -w[ids[:, 0], :, at]
    y = torch.empty(tokens, n, dtype=types[1], device="cuda")
    ones = torch.ones(tokens, 1, device="cuda")
    qmm.qmm_experts_down_q4_0(dev(b), dev(x[pairs], types[0]), y, dev(ids.astype(np.int32)), ones, dev(starts), dev(pairs), n, k)
    limit = 2.0 ** -10 + (2.0 ** -24 if types[1] is F32 else 2.0 ** -8)
    assert (np.abs(y.double().cpu().numpy() - want) <= limit * np.abs(want)).all()
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


@pytest.mark.parametrize("tokens,experts,types", [(3, 64, t) for t in ((F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16))] +
                         [(90, 4, t) for t in ((F32, F32), (F32, BF16), (BF16, F32))], ids=str)
def test_sums_of_a_block_are_whole(qmm, types, tokens, experts):
    """v, -v and -1 in a block of one code, v of 17 bits, in the streaming form: integers to
    2^20 whose sum, the code, is exact in 24 bits; times the scale exact too, but for the
    result's rounding.  (The tile form adds products of weights: 14 bits below each of v's
    17, so that addends of 2^17 |w| leave 2^-6 |w| in 24 bits.)"""
    rng = np.random.default_rng(tokens + experts)
    n, k = 48, 256
    b = ref.blocks(rng, experts, n, k)
    row = b.reshape(experts, n, k // 32, 18)
    row[:, :, 0, 2:] = rng.integers(0, 16, (experts, n, 1)) * 17
    ids = rng.integers(0, experts, (tokens, 1))
    starts, pairs = ref.plan_of(ids, experts)
    x = np.zeros((tokens, k), dtype=np.float32)
    for t in range(tokens):
        at = rng.permutation(32)[:3]
        v = 512 * int(rng.integers(128, 256))
        x[t, at] = v, -v, -1
    w, _ = ref.matrix(b)
    want = -w[ids[:, 0], :, 0]
    y = torch.empty(tokens, n, dtype=types[1], device="cuda")
    ones = torch.ones(tokens, 1, device="cuda")
    qmm.qmm_experts_down_q4_0(dev(b), dev(x[pairs], types[0]), y, dev(ids.astype(np.int32)), ones, dev(starts), dev(pairs), n, k)
    limit = 0.0 if types[1] is F32 else 2.0 ** -8
    assert (np.abs(y.double().cpu().numpy() - want) <= limit * np.abs(want)).all()
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


@pytest.mark.parametrize("y_type", [F32, BF16], ids=str)
@pytest.mark.parametrize("tokens,experts", [(3, 64), (3, 4), (40, 16), (90, 4)])
@pytest.mark.parametrize("k", [256, 288])
def test_bf16_rows_of_any_range(qmm, y_type, tokens, experts, k):
    """Rows whose largest value, 1e30, meets weights of 0, beside values of 1 and of 1e-30; in all
    forms.  Bounds: those of exact products of the other values, and the result's rounding."""
    rng = np.random.default_rng(tokens + experts + k)
    n, topk = 40, 2
    ids = np.argsort(rng.random((tokens, experts)), axis=1)[:, :topk]
    starts, pairs = ref.plan_of(ids, experts)
    weights = rng.random((tokens, topk)).astype(np.float32)
    b = ref.blocks(rng, experts, n, k)
    row = b.reshape(experts, n, k // 32, 18)
    row[:, :, 1, 2 + 5] = row[:, :, 1, 2 + 5] & 0xF0 | 8  # value 37 of each row of weights is 0
    h = rng.standard_normal((tokens * topk, k)).astype(np.float32)
    h[::3] *= 1e-30
    h[:, 37] = 0
    h = torch.from_numpy(h).bfloat16()
    want, limit = ref.experts_down(h.double().numpy(), b, ids, weights, starts, pairs, True, False)
    h[:, 37] = 1e30
    y = torch.empty(tokens, n, dtype=y_type, device="cuda")
    qmm.qmm_experts_down_q4_0(dev(b), h.cuda(), y, dev(ids.astype(np.int32)), dev(weights), dev(starts), dev(pairs), n, k)
    limit = limit + (2.0 ** -8 if y_type is BF16 else 2.0 ** -24) * (np.abs(want) + limit)
    assert (np.abs(y.double().cpu().numpy() - want) <= limit).all()
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


@pytest.mark.parametrize("types", [(BF16, BF16), (F32, BF16)], ids=str)
@pytest.mark.parametrize("size", [(3, 64, 4, 130, 512), (16, 8, 2, 64, 1024), (70, 4, 2, 40, 256), (300, 8, 4, 260, 256), (257, 16, 8, 64, 288),
                                  (200, 6, 3, 129, 2080), (33, 4, 2, 96, 2048)], ids=str)
def test_bf16_results_are_rounded_once(qmm, size, types):
    """Both products within the bounds of fp32 results, and half a step of bf16."""
    tokens, experts, topk, n, k = size
    rng = np.random.default_rng(sum(size))
    ids = np.argsort(rng.random((tokens, experts)), axis=1)[:, :topk]
    starts, pairs = ref.plan_of(ids, experts)
    bg, bu = ref.blocks(rng, experts, n, k), ref.blocks(rng, experts, n, k)

    def near(got, want, limit):
        limit = limit + 2.0 ** -8 * (np.abs(want) + limit)
        assert (np.abs(got.double().cpu().numpy() - want) <= limit).all()

    x = torch.from_numpy(rng.standard_normal((tokens, k)).astype(np.float32)).to(types[0])
    h = torch.empty(tokens * topk, n, dtype=BF16, device="cuda")
    qmm.qmm_experts_geglu_q4_0(dev(bg), dev(bu), x.cuda(), h, dev(starts), dev(pairs), topk, n, k)
    near(h, *ref.experts_geglu(x.double().numpy(), bg, bu, starts, pairs, topk, True, False))
    x = torch.from_numpy(rng.standard_normal((tokens * topk, k)).astype(np.float32)).to(types[0])
    weights = rng.standard_normal((tokens, topk)).astype(np.float32)
    y = torch.empty(tokens, n, dtype=BF16, device="cuda")
    qmm.qmm_experts_down_q4_0(dev(bg), x.cuda(), y, dev(ids.astype(np.int32)), dev(weights), dev(starts), dev(pairs), n, k)
    near(y, *ref.experts_down(x.double().numpy(), bg, ids, weights, starts, pairs, True, False))
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


@pytest.mark.parametrize("types", [(BF16, BF16), (F32, F32)], ids=str)
@pytest.mark.parametrize("tokens,experts", [(3, 64), (90, 4)])
@pytest.mark.parametrize("k", [256, 288])
def test_scales_of_both_signs(qmm, types, tokens, experts, k):
    """Scales as quantizers leave them, negative where the largest value is positive, and 0 among them."""
    rng = np.random.default_rng(tokens + experts + k)
    n, topk = 72, 2
    b = ref.blocks(rng, experts, n, k)
    row = b.reshape(experts, n, k // 32, 18)
    row[..., 1] ^= (rng.integers(0, 2, row.shape[:3]) * 128).astype(np.uint8)  # binary16's sign
    row[:, 5::7, 2, :2] = 0
    ids = np.argsort(rng.random((tokens, experts)), axis=1)[:, :topk]
    starts, pairs = ref.plan_of(ids, experts)
    weights = rng.standard_normal((tokens, topk)).astype(np.float32)
    h = torch.from_numpy(rng.standard_normal((tokens * topk, k)).astype(np.float32)).to(types[0])
    want, limit = ref.experts_down(h.double().numpy(), b, ids, weights, starts, pairs, True, False)
    y = torch.empty(tokens, n, dtype=types[1], device="cuda")
    qmm.qmm_experts_down_q4_0(dev(b), h.cuda(), y, dev(ids.astype(np.int32)), dev(weights), dev(starts), dev(pairs), n, k)
    limit = limit + (2.0 ** -8 if types[1] is BF16 else 2.0 ** -24) * (np.abs(want) + limit)
    assert (np.abs(y.double().cpu().numpy() - want) <= limit).all()
    assert qmm.qmm_get_device_error() == qmm.QMM_OK
