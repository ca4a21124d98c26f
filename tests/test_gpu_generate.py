"""The generation loop: the calls work together, and each step's attention is
that of the cache it left behind."""
import numpy as np
import pytest

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


def check_attention(g):
    """The last step's outputs against the cache's contents, in 64 bits."""
    arrays = [t.cpu().numpy() for t in (g.cache.k_codes, g.cache.k_scales, g.cache.v_codes, g.cache.v_scales)]
    last = g.last
    want = ref.attention(last["q"].double().cpu().numpy(), *arrays, g.table.cpu().numpy(), last["q_start"].tolist(),
                         g.kv_len.tolist(), g.layer.head_dim ** -0.5, True, 0)
    out = last["out"]
    limit, _ = ref.attention_limits(*want, bf16=out.dtype == torch.bfloat16)
    assert (np.abs(out.float().cpu().numpy() - want[0]) <= limit).all()


@pytest.mark.parametrize("prompts", [[[5]], [[1, 2, 3], [4] * 40, []], [list(range(100)), [9, 8], list(range(33))]])
def test_prompts_and_steps(gen, prompts):
    from block_quantized_matmul_gguf_gb300 import qmm
    layer = gen.Layer(hidden=256, heads=4, kv_heads=2, head_dim=64, vocab=512, seed=3)
    g = gen.Generator(layer, len(prompts))
    tokens = prompts
    total = [0] * len(prompts)
    for _ in range(4):
        new = g.step(tokens)
        total = [n + len(t) for n, t in zip(total, tokens)]
        assert g.kv_len.tolist() == total
        assert all(0 <= t < layer.vocab for t in new)
        check_attention(g)
        tokens = [[t] for t in new]
    assert qmm.qmm_get_device_error() == qmm.QMM_OK
    again = gen.Generator(layer, len(prompts)).run(prompts, 4)
    assert again == gen.Generator(layer, len(prompts)).run(prompts, 4)


def test_masks_and_biases_steer_the_tokens(gen):
    layer = gen.Layer(hidden=256, heads=4, kv_heads=1, head_dim=128, vocab=512, seed=4)
    prompts = [[1, 2], [3]]
    words = torch.zeros((2, 16), dtype=torch.int32)
    words[:, 3] = 0b1010  # tokens 97 and 99
    made = gen.Generator(layer, 2).run(prompts, 6, allowed=words.cuda())
    assert {t for m in made for t in m} <= {97, 99}
    made = gen.Generator(layer, 2).run(prompts, 3, repetition=1.0, frequency=0.0, presence=0.0, bias={300: 1e6})
    assert all(t == 300 for m in made for t in m)
    with pytest.raises(RuntimeError):
        gen.Generator(layer, 1, num_pages=1).run([[1] * 40], 1)
