"""Weights of experts whose scores are small: their quotients stay what the formula says."""
import numpy as np
import pytest

import experts_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qmm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_quantized_matmul_gguf_gb300 import build, qmm
    build.build_library()
    return qmm


def weights_of(x, ids, score, renormalize, scale):
    """From the scores' logarithms, in 64 bits."""
    log = -np.logaddexp(0, -x) if score == "sigmoid" else x - np.logaddexp.reduce(x, 1, keepdims=True)
    log = np.take_along_axis(log, ids, 1)
    if renormalize:
        log = log - np.logaddexp.reduce(log, 1, keepdims=True)
    return np.exp(log) * scale


def run(qmm, logits, topk, bias=None, **kw):
    tokens, experts = logits.shape
    i32 = dict(dtype=torch.int32, device="cuda")
    ids, weights = torch.empty(tokens, topk, **i32), torch.empty(tokens, topk, device="cuda")
    qmm.qmm_route(logits.cuda(), ids, weights, torch.empty(experts + 1, **i32), torch.empty(tokens * topk, **i32),
                  bias=None if bias is None else bias.cuda(), **kw)
    assert qmm.qmm_get_device_error() == qmm.QMM_OK
    return ids.cpu().numpy(), weights.double().cpu().numpy()


def near(got, want):
    # ref.WEIGHT: a quotient's roundings and those of differences of logits to some
    # 100; below the smallest normal number two steps of the smallest there is, 2^-149
    assert (np.abs(got - want) <= ref.WEIGHT * want + 2.0 ** -148).all(), (got[:2], want[:2])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("level", [0.0, -30.0, -63.0, -64.5, -80.0, -87.5, -90.0, -95.0, -104.0, -200.0, -650.0, 90.0])
@pytest.mark.parametrize("spread", [0.0, 1.5, 20.0])
def test_sigmoid_logits_of_any_size(qmm, level, spread, renormalize, dtype):
    rng = np.random.default_rng(int(-level) + 100)
    logits = torch.from_numpy((level + spread * rng.standard_normal((70, 48))).astype(np.float32))
    if dtype == "bf16":
        logits = logits.bfloat16()
    kw = dict(score="sigmoid", renormalize=renormalize, scale=2.5)
    ids, weights = run(qmm, logits, 6, **kw)
    want = ref.route(logits.double().numpy(), None, 6, "sigmoid")[0]
    assert np.array_equal(ids, want)
    near(weights, weights_of(logits.double().numpy(), ids, "sigmoid", renormalize, 2.5))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("level", [-10.0, -80.0, -90.0, -110.0, -300.0, -600.0])
def test_a_bias_chooses_experts_far_below_the_largest(qmm, level, groups, score):
    rng = np.random.default_rng(int(-level))
    tokens, experts, topk = 40, 32, 4
    x = rng.standard_normal((tokens, experts))
    x[:, experts // 4:] += level
    bias = torch.zeros(experts)
    bias[:experts // 4] = -2.0  # the likely ones are hidden
    bias[experts // 4:] = torch.linspace(0.3, 0.7, experts - experts // 4)
    logits = torch.from_numpy(x.astype(np.float32))
    kw = dict(score=score, groups=groups, group_topk=1 if groups > 1 else 1)
    ids, weights = run(qmm, logits, topk, bias, **kw)
    assert (ids >= experts // 4).all()
    near(weights, weights_of(logits.double().numpy(), ids, score, True, 1.0))
    assert (np.abs(weights.sum(1) - 1) < 2.0 ** -16).all()


def test_scores_of_zero_have_weights_of_zero(qmm):
    """Scores that are 0 in 64 bits: logits of -inf or the type's lowest, and some 745 below."""
    lowest = torch.finfo(torch.float32).min
    logits = torch.full((5, 16), -1000.0)
    logits[1], logits[2] = -float("inf"), lowest
    logits[3, :2], logits[4, 1:] = 0.0, -float("inf")
    bias = torch.linspace(0, -5, 16)
    ids, weights = run(qmm, logits, 4, score="sigmoid", bias=bias)
    assert (weights[:3] == 0).all() and (weights[3] == [0.5, 0.5, 0, 0]).all() and (weights[4] == 0).all()
    hide = torch.zeros(16)
    hide[:4] = -float("inf")
    logits = torch.full((3, 16), -800.0)
    logits[:, 0] = 0.0
    logits[1, 4:], logits[2, 4:] = -float("inf"), lowest
    ids, weights = run(qmm, logits, 4, score="softmax", bias=hide)
    assert (ids >= 4).all() and (weights == 0).all()
