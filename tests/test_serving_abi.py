"""Argument checks of the serving entry points (cache, attention, logits):
every refusal happens before any CUDA call, so these run without a GPU.
Pointers are fake values far apart, never dereferenced."""
import ctypes

import pytest

from block_quantized_matmul_gguf_gb300 import build, qmm

M = 1 << 24
OK, NULL, SHAPE = qmm.QMM_OK, qmm.QMM_ERR_NULL, qmm.QMM_ERR_SHAPE
ALIGN, UNSUPPORTED = qmm.QMM_ERR_ALIGN, qmm.QMM_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return qmm.load()


def cache(**kw):
    f = dict(k_codes=1 * M, k_scales=2 * M, v_codes=3 * M, v_scales=4 * M, num_pages=8, page_size=16,
             kv_heads=2, head_dim=64)
    f.update(kw)
    return qmm.KvQ4_0(**f)


def ref(s):
    return ctypes.addressof(s)


BAD_CACHES = [
    (dict(k_codes=None), NULL), (dict(k_scales=None), NULL), (dict(v_codes=None), NULL),
    (dict(v_scales=None), NULL), (dict(num_pages=0), SHAPE), (dict(kv_heads=0), SHAPE),
    (dict(head_dim=0), SHAPE), (dict(page_size=0), SHAPE), (dict(head_dim=96), UNSUPPORTED),
    (dict(head_dim=512), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED),
    (dict(page_size=2048), UNSUPPORTED), (dict(num_pages=1 << 26), UNSUPPORTED),
    (dict(num_pages=1 << 40), UNSUPPORTED), (dict(k_codes=M + 8), ALIGN), (dict(v_scales=4 * M + 4), ALIGN),
]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_cache_checks_are_those_of_every_call(lib, kw, status):
    c = cache(**kw)
    assert lib.qmm_kv_append_q4_0(ref(c), 5 * M, 128, 6 * M, 128, 0, 7 * M, 4, None) == status
    assert lib.qmm_kv_read_q4_0(ref(c), 7 * M, 4, 5 * M, 6 * M, None) == status
    assert lib.qmm_attn_q4_0(ref(c), ref(attn()), None) == status


def test_plan_checks(lib):
    good = [5 * M, 6 * M, 4, 7 * M, 10, 8 * M, 6, 16, 9 * M, 10 * M, 11 * M, 12 * M, 32, 13 * M, None]

    def call(**at):
        a = list(good)
        for k, v in at.items():
            a[int(k[1:])] = v
        return lib.qmm_kv_plan(*a)

    for i in (0, 1, 3, 5, 8, 9, 10, 11, 13):
        assert call(**{f"_{i}": None}) == NULL
    assert call(_2=0) == SHAPE and call(_4=-1) == SHAPE and call(_6=0) == SHAPE
    assert call(_7=0) == SHAPE and call(_12=-1) == SHAPE
    assert call(_7=24) == UNSUPPORTED and call(_2=16385) == UNSUPPORTED and call(_4=1 << 31) == UNSUPPORTED
    assert call(_0=5 * M + 2) == ALIGN and call(_10=11 * M + 4) == ALIGN
    assert call(_8=5 * M) == UNSUPPORTED          # q_start over cached
    assert call(_9=9 * M + 8) == UNSUPPORTED      # kv_len over q_start
    assert call(_5=7 * M + 16) == UNSUPPORTED     # table over free_pages


def test_append_and_read_checks(lib):
    c = cache()

    def app(k=5 * M, ks=128, v=6 * M, vs=128, t=0, slots=7 * M, n=4):
        return lib.qmm_kv_append_q4_0(ref(c), k, ks, v, vs, t, slots, n, None)

    assert lib.qmm_kv_append_q4_0(None, 5 * M, 128, 6 * M, 128, 0, 7 * M, 4, None) == NULL
    assert app(n=0) == OK and app(n=0, k=None) == OK
    assert app(k=None) == NULL and app(v=None) == NULL and app(slots=None) == NULL
    assert app(n=-1) == SHAPE and app(ks=127) == SHAPE and app(vs=64) == SHAPE and app(t=2) == SHAPE
    assert app(n=(1 << 30) + 1) == UNSUPPORTED
    assert app(k=5 * M + 2) == ALIGN and app(slots=7 * M + 4) == ALIGN and app(t=1, k=5 * M + 1) == ALIGN
    assert app(k=3 * M) == UNSUPPORTED and app(slots=2 * M) == UNSUPPORTED

    def read(slots=7 * M, n=4, k=5 * M, v=6 * M):
        return lib.qmm_kv_read_q4_0(ref(c), slots, n, k, v, None)

    assert read(n=0) == OK and read(n=-1) == SHAPE
    assert read(slots=None) == NULL and read(k=None, v=None) == NULL
    assert read(k=5 * M + 2) == ALIGN and read(slots=7 * M + 2) == ALIGN
    assert read(k=5 * M, v=5 * M + 64) == UNSUPPORTED and read(k=M) == UNSUPPORTED and read(v=7 * M) == UNSUPPORTED


def attn(**kw):
    f = dict(q=5 * M, q_stride=256, q_type=0, out=6 * M, out_stride=256, out_type=0, lse=7 * M, table=8 * M,
             table_width=4, q_start=9 * M, kv_len=10 * M, batch=3, total_q=5, max_q=2, heads=4, scale=0.125,
             causal=1, window=0, workspace=1 << 40, workspace_bytes=1 << 30)
    f.update(kw)
    return qmm.AttnArgs(**f)


@pytest.mark.parametrize("kw,status", [
    (dict(total_q=0), OK), (dict(total_q=0, q=None), OK),
    (dict(q=None), NULL), (dict(out=None), NULL), (dict(table=None), NULL), (dict(q_start=None), NULL),
    (dict(kv_len=None), NULL), (dict(batch=0), SHAPE), (dict(total_q=-1), SHAPE), (dict(max_q=0), SHAPE),
    (dict(heads=0), SHAPE), (dict(heads=3), SHAPE), (dict(table_width=0), SHAPE), (dict(window=-1), SHAPE),
    (dict(window=8, causal=0), SHAPE), (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE),
    (dict(q_type=2), SHAPE), (dict(out_type=-1), SHAPE), (dict(q_stride=255), SHAPE),
    (dict(out_stride=128), SHAPE), (dict(batch=16385), UNSUPPORTED), (dict(total_q=(1 << 30) + 1), UNSUPPORTED),
    (dict(heads=1026, q_stride=1026 * 64, out_stride=1026 * 64), UNSUPPORTED),
    (dict(q=5 * M + 2), ALIGN), (dict(q_type=1, q=5 * M + 1), ALIGN), (dict(out=6 * M + 2), ALIGN),
    (dict(lse=7 * M + 2), ALIGN), (dict(kv_len=10 * M + 1), ALIGN),
    (dict(out=5 * M), UNSUPPORTED), (dict(lse=6 * M + 16), UNSUPPORTED), (dict(out=3 * M), UNSUPPORTED),
    (dict(lse=8 * M), UNSUPPORTED),
])
def test_attention_checks(lib, kw, status):
    assert lib.qmm_attn_q4_0(ref(cache()), ref(attn(**kw)), None) == status


def test_attention_needs_a_cache_and_arguments(lib):
    assert lib.qmm_attn_q4_0(None, ref(attn()), None) == NULL
    assert lib.qmm_attn_q4_0(ref(cache()), None, None) == NULL
    assert lib.qmm_attn_q4_0_workspace_bytes(None, 4) == 0
    assert lib.qmm_attn_q4_0_workspace_bytes(ref(cache()), 3) == 0


def logits(**kw):
    f = dict(logits=1 * M, logits_stride=1000, out=2 * M, out_stride=1000, rows=3, vocab=1000, history=3 * M,
             hist_start=4 * M, history_len=50, prompt_len=5 * M, repetition=6 * M, frequency=7 * M,
             presence=8 * M, bias_ids=9 * M, bias_values=10 * M, bias_start=11 * M, bias_len=9, allowed=12 * M)
    f.update(kw)
    return qmm.LogitsArgs(**f)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), NULL), (dict(out=None), NULL), (dict(hist_start=None), NULL), (dict(history=None), NULL),
    (dict(bias_values=None), NULL), (dict(bias_start=None), NULL), (dict(bias_ids=None), NULL),
    (dict(rows=0), SHAPE), (dict(vocab=0), SHAPE), (dict(logits_stride=999), SHAPE), (dict(out_stride=1), SHAPE),
    (dict(history_len=-1), SHAPE), (dict(bias_len=-1), SHAPE), (dict(rows=65536), UNSUPPORTED),
    (dict(vocab=(1 << 31) - 1, logits_stride=1 << 31, out_stride=1 << 31), UNSUPPORTED),
    (dict(logits=M + 2), ALIGN), (dict(allowed=12 * M + 1), ALIGN), (dict(presence=8 * M + 2), ALIGN),
    (dict(out=M, out_stride=1001), UNSUPPORTED), (dict(out=M + 4000), UNSUPPORTED),
    (dict(out=3 * M), UNSUPPORTED), (dict(out=12 * M), UNSUPPORTED),
])
def test_logits_checks(lib, kw, status):
    assert lib.qmm_logits_adjust(ref(logits(**kw)), None) == status
    assert lib.qmm_logits_adjust(None, None) == NULL


def test_index_status_has_its_text(lib):
    assert "outside" in qmm.status_string(qmm.QMM_ERR_INDEX)


def test_packed_arguments_have_the_structs_layout():
    """The binding packs the argument structs; each field must land where the
    declared struct has it."""
    for packer, cls in ((qmm._ATTN_ARGS, qmm.AttnArgs), (qmm._LOGITS_ARGS, qmm.LogitsArgs)):
        values = list(range(1, len(cls._fields_) + 1))
        raw = packer.pack(*values)
        assert ctypes.sizeof(cls) - 8 < len(raw) <= ctypes.sizeof(cls)
        s = cls.from_buffer_copy(raw.ljust(ctypes.sizeof(cls), b"\0"))
        assert [getattr(s, name) for name, _ in cls._fields_] == values
