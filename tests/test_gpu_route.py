"""Routing to experts: ids, starts and pairs equal to the 64-bit reference's,
weights within the bound derived in experts_ref."""
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


def outputs(tokens, experts, topk):
    i32 = dict(dtype=torch.int32, device="cuda")
    return [torch.full((tokens, topk), -9, **i32), torch.full((tokens, topk), -9.0, device="cuda"),
            torch.full((experts + 1,), -9, **i32), torch.full((tokens * topk,), -9, **i32)]


def run(qmm, logits, topk, bias=None, **kw):
    out = outputs(logits.shape[0], logits.shape[1], topk)
    qmm.qmm_route(logits.cuda(), *out, bias=None if bias is None else bias.cuda(), **kw)
    return [t.cpu().numpy() for t in out]


def check(got, want):
    assert np.array_equal(got[0], want[0]), "ids"
    assert np.array_equal(got[2], want[2]), "expert_start"
    assert np.array_equal(got[3], want[3]), "pairs"
    finite = np.isfinite(want[1])
    assert np.array_equal(np.isnan(got[1]), np.isnan(want[1]))
    assert (np.abs(got[1] - want[1])[finite] <= ref.WEIGHT * np.abs(want[1])[finite] + 1e-37).all(), "weights"


CASES = [  # tokens, experts, topk, groups, kept, best
    (1, 1, 1, 1, 1, 1), (1, 64, 8, 1, 1, 1), (2, 33, 32, 1, 1, 1), (63, 64, 6, 1, 1, 1), (64, 128, 8, 1, 1, 1),
    (65, 31, 3, 1, 1, 1), (200, 60, 4, 4, 2, 1), (129, 256, 8, 8, 4, 2), (1000, 96, 7, 3, 1, 2), (77, 512, 10, 32, 5, 1),
    (50, 1024, 32, 1, 1, 1), (300, 1024, 8, 16, 3, 2), (4099, 160, 6, 8, 3, 2), (17000, 40, 2, 1, 1, 1),
]


@pytest.mark.parametrize("tokens,experts,topk,groups,kept,best", CASES)
@pytest.mark.parametrize("score,bias,dtype", [("softmax", False, "f32"), ("sigmoid", True, "f32"),
                                              ("softmax", True, "bf16"), ("sigmoid", False, "bf16")])
def test_choice_and_order(qmm, tokens, experts, topk, groups, kept, best, score, bias, dtype):
    g = torch.Generator().manual_seed(tokens + experts + topk)
    logits = torch.randn(tokens, experts, generator=g) * 2
    if dtype == "bf16":
        logits = logits.bfloat16()  # equal logits are common
    b = torch.randn(experts, generator=g) * 0.1 if bias else None
    kw = dict(score=score, groups=groups, group_topk=kept, group_best=best, scale=2.5)
    want = ref.route(logits.double().numpy(), None if b is None else b.double().numpy(), topk, **kw)
    check(run(qmm, logits, topk, b, **kw), want)
    again = run(qmm, logits, topk, b, **kw)
    check(again, want)
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,best", [(1, 1), (4, 2)])
def test_scores_too_near_for_32_bits(qmm, score, groups, best):
    """Biases that put experts' values 1e-9 to 1e-7 apart, in an order that fp32 cannot see."""
    rng = np.random.default_rng(7)
    tokens, experts, topk = 96, 64, 6
    logits = rng.standard_normal(experts).astype(np.float32)
    x = logits.astype(np.float64)
    s = 1 / (1 + np.exp(-x)) if score == "sigmoid" else np.exp(x) / np.exp(x).sum()
    # as near as fp32 biases come: their own spacing keeps the values apart
    bias = (0.5 - s + rng.permutation(experts) * 1e-9).astype(np.float32)
    rows = np.repeat(logits[None], tokens, 0)
    rows[::2] = rng.standard_normal((tokens // 2, experts))  # ordinary ones among them
    kw = dict(score=score, groups=groups, group_topk=max(1, groups // 2), group_best=best)
    want = ref.route(rows.astype(np.float64), bias.astype(np.float64), topk, **kw)
    check(run(qmm, torch.from_numpy(rows), topk, torch.from_numpy(bias), **kw), want)


def test_equal_scores_go_to_the_lowest_index(qmm):
    logits = torch.zeros(70, 96)
    logits[1, 5], logits[2, ::2] = -0.0, 1.0
    for kw in (dict(), dict(groups=4, group_topk=2), dict(groups=4, group_topk=2, group_best=2)):
        for bias in (None, torch.full((96,), 0.25)):
            want = ref.route(logits.numpy(), None if bias is None else bias.numpy(), 5, "softmax", **kw)
            check(run(qmm, logits, 5, bias, score="softmax", **kw), want)
            assert want[0][0].tolist() == [0, 1, 2, 3, 4]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_masked_and_odd_logits(qmm, score, biased):
    """Experts and whole rows at -inf or the type's lowest value, and NaN, which comes last."""
    inf = float("inf")
    logits = torch.randn(8, 40, generator=torch.Generator().manual_seed(1))
    logits[0, 3:] = -inf
    logits[1] = -inf
    logits[2, ::3] = torch.finfo(torch.float32).min
    logits[3] = torch.finfo(torch.float32).min
    logits[4, 7] = float("nan")
    logits[5] = float("nan")
    bias = torch.linspace(-0.2, 0.2, 40) if biased else None
    for renormalize in (True, False):
        kw = dict(score=score, renormalize=renormalize)
        want = ref.route(logits.double().numpy(), None if bias is None else bias.double().numpy(), 4, **kw)
        got = run(qmm, logits, 4, bias, **kw)
        check([g[:4] if i < 2 else g for i, g in enumerate(got)][:2] + got[2:],
              [w[:4] if i < 2 else w for i, w in enumerate(want)][:2] + list(want[2:]))
        assert np.array_equal(got[0], want[0])
        assert sorted(got[3].tolist()) == list(range(32))
    # a bias that masks
    hide = torch.zeros(40)
    hide[::2] = -inf
    want = ref.route(logits[6:].double().numpy(), hide.double().numpy(), 9, score)
    check(run(qmm, logits[6:], 9, hide, score=score), want)
    assert (want[0] % 2 == 1).all()


@pytest.mark.parametrize("tokens,count", [(5, 0), (64, 1), (65, 64), (1000, 700), (300, 300)])
def test_tokens_that_are_not_there(qmm, tokens, count):
    logits = torch.randn(tokens, 32, generator=torch.Generator().manual_seed(tokens))
    n = torch.tensor([count], dtype=torch.int32).cuda()
    want = ref.route(logits.numpy(), None, 4, "softmax", count=count)
    check(run(qmm, logits, 4, count=n), want)
    assert qmm.qmm_get_device_error() == qmm.QMM_OK
    for odd in (-1, tokens + 1):
        n.fill_(odd)
        check(run(qmm, logits, 4, count=n), ref.route(logits.numpy(), None, 4, "softmax", count=odd))
        assert qmm.qmm_get_device_error() == qmm.QMM_ERR_INDEX


@pytest.mark.parametrize("tokens", [40, 500])
def test_strides_streams_and_graphs(qmm, tokens):
    wide = torch.randn(tokens, 70, generator=torch.Generator().manual_seed(3)).cuda()
    logits = wide[:, 3:67]
    want = ref.route(logits.cpu().numpy(), None, 8, "softmax")
    side = torch.cuda.Stream()
    out = outputs(tokens, 64, 8)
    torch.cuda.synchronize()
    qmm.qmm_route(logits, *out, stream=side)
    side.synchronize()
    check([t.cpu().numpy() for t in out], want)
    # captured, then replayed on other logits and another count
    n = torch.tensor([tokens], dtype=torch.int32).cuda()
    ws = qmm.route_workspace(tokens, 64)
    out = outputs(tokens, 64, 8)
    with torch.cuda.stream(side):
        qmm.qmm_route(logits, *out, count=n, workspace=ws)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        qmm.qmm_route(logits, *out, count=n, workspace=ws)
    wide.copy_(torch.randn(tokens, 70, generator=torch.Generator().manual_seed(4)))
    n.fill_(tokens - 7)
    graph.replay()
    torch.cuda.synchronize()
    check([t.cpu().numpy() for t in out], ref.route(logits.cpu().numpy(), None, 8, "softmax", count=tokens - 7))


def test_nothing_to_do_and_refusals(qmm):
    out = outputs(0, 8, 2)
    qmm.qmm_route(torch.empty(0, 8).cuda(), *out)
    logits = torch.zeros(3, 8).cuda()
    with pytest.raises(ValueError):
        qmm.qmm_route(logits.half(), *outputs(3, 8, 2))
    with pytest.raises(ValueError):
        qmm.qmm_route(logits, *outputs(4, 8, 2))
    with pytest.raises(ValueError):
        qmm.qmm_route(logits, *outputs(3, 8, 2), score="tanh")
    with pytest.raises(ValueError):
        qmm.qmm_route(logits, *outputs(3, 8, 2), bias=torch.zeros(7).cuda())
    with pytest.raises(qmm.QmmError):
        qmm.qmm_route(logits, *outputs(3, 8, 2), groups=3)
