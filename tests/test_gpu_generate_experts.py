"""The generation loop with rotated queries and keys and with experts: each
step's attention is that of the cache it left behind, its keys are those of
their positions, and its experts' outputs are those of its own routing, in
64 bits."""
import numpy as np
import pytest

import experts_ref
import serving_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gen():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_quantized_matmul_gguf_gb300 import build, generate
    build.build_library()
    return generate


SIZES = dict(hidden=256, heads=4, kv_heads=2, head_dim=64, vocab=512, seed=3)
PROMPTS = [[[5]], [[1, 2, 3], [4] * 40, []], [list(range(100)), [9, 8], list(range(33))]]


def host(t):
    return t.cpu().numpy()


def check_attention(g):
    last = g.last
    arrays = [host(t) for t in (g.cache.k_codes, g.cache.k_scales, g.cache.v_codes, g.cache.v_scales)]
    want = ref.attention(last["q"].double().cpu().numpy(), *arrays, host(g.table), last["q_start"].tolist(),
                         g.kv_len.tolist(), g.layer.head_dim ** -0.5, True, 0)
    limit, _ = ref.attention_limits(*want, bf16=last["out"].dtype == torch.bfloat16)
    assert (np.abs(last["out"].float().cpu().numpy() - want[0]) <= limit).all()


def check_experts(g):
    layer, r = g.layer, {k: v.double().cpu().numpy() if v.is_floating_point() else host(v) for k, v in g.routed.items()}
    bf16 = g.routed["x"].dtype == torch.bfloat16
    ids, weights, starts, pairs = experts_ref.route(r["logits"], None, layer.topk, "softmax")
    assert np.array_equal(r["ids"], ids) and np.array_equal(r["starts"], starts) and np.array_equal(r["pairs"], pairs)
    assert (np.abs(r["weights"] - weights) <= experts_ref.WEIGHT * weights + 1e-30).all()

    def blocks(w, n, k):
        return host(w).reshape(layer.experts, n, k // 32 * 18)

    width, hidden = layer.expert_width, layer.hidden
    h, limit = experts_ref.experts_geglu(r["x"], blocks(layer.wg, width, hidden), blocks(layer.wu, width, hidden),
                                         starts, pairs, layer.topk, not bf16, not bf16)
    assert (np.abs(r["h"] - h) <= limit).all()
    y, limit = experts_ref.experts_down(r["h"], blocks(layer.wd, hidden, width), ids, r["weights"].astype(np.float32),
                                        starts, pairs, not bf16, not bf16)
    assert (np.abs(r["y"] - y) <= limit).all()


@pytest.mark.parametrize("prompts", PROMPTS)
@pytest.mark.parametrize("more", [dict(rope=10000.0), dict(experts=8), dict(rope=500.0, experts=40, topk=4)], ids=str)
def test_prompts_and_steps(gen, prompts, more):
    from block_quantized_matmul_gguf_gb300 import qmm
    layer = gen.Layer(**SIZES, **more)
    g = gen.Generator(layer, len(prompts))
    tokens, total = prompts, [0] * len(prompts)
    for _ in range(4):
        new = g.step(tokens)
        total = [n + len(t) for n, t in zip(total, tokens)]
        assert g.kv_len.tolist() == total and all(0 <= t < layer.vocab for t in new)
        check_attention(g)
        if layer.experts:
            check_experts(g)
        tokens = [[t] for t in new]
    assert qmm.qmm_get_device_error() == qmm.QMM_OK
    again = gen.Generator(layer, len(prompts)).run(prompts, 4)
    assert again == gen.Generator(layer, len(prompts)).run(prompts, 4)


def test_keys_lie_where_their_positions_turn_them(gen):
    """One request's keys against another layer's without a rotation: the same key, turned back in 64 bits."""
    from block_quantized_matmul_gguf_gb300 import qmm
    prompt = list(range(7, 60))
    caches = []
    for rope in (None, 10000.0):
        layer = gen.Layer(**SIZES, rope=rope)
        g = gen.Generator(layer, 1)
        g.step([prompt])
        k = torch.empty((len(prompt), layer.kv_heads, layer.head_dim), device="cuda")
        qmm.qmm_kv_read_q4_0(g.cache, g.last["slots"], k, None)
        caches.append(k.double().cpu().numpy())
        q = g.last["q"].double().cpu().numpy()
        caches.append(q)
    plain, q, turned, q_turned = caches
    half = plain.shape[-1] // 2
    angle = np.arange(len(prompt))[:, None] * 10000.0 ** (np.arange(half) * (-2.0 / plain.shape[-1]))
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]

    def turn(v):
        a, b = v[..., :half], v[..., half:]
        return np.concatenate([a * c - b * s, a * s + b * c], -1)

    # q: projected to fp32 and rotated in fp32: the table, two products and a sum, under 8 half steps
    size = np.concatenate([np.hypot(q[..., :half], q[..., half:])] * 2, -1)
    assert (np.abs(q_turned - turn(q)) <= 2.0 ** -21 * size + 1e-30).all()
    # k: a Q4_0 code is off by its scale at most (the largest of a block's 32 values is 8 scales, codes end at
    # +7), on both sides; a turn takes both values of a pair with |c| + |s| <= sqrt 2
    def step(v):
        d = np.abs(v.reshape(*v.shape[:-1], -1, 32)).max(-1) / 7.0  # a block of zeros has none
        return np.repeat(d, 32, -1)
    e = step(plain)
    e = np.sqrt(2.0) * np.maximum(np.concatenate([e[..., half:], e[..., :half]], -1), e)
    assert (np.abs(turned - turn(plain)) <= e + step(turned) + 1e-6).all()
    assert np.abs(turned - plain).max() > 10 * (e + step(turned)).min()  # and they are turned


def test_defaults_have_no_rotation_and_no_experts(gen):
    g = gen.Generator(gen.Layer(**SIZES), 1)
    g.step([[1, 2, 3]])
    assert g.rotations is None and not hasattr(g, "routed")
