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
