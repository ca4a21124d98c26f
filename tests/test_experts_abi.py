"""Argument checks of the rotation, the routing and the experts' products:
every refusal happens before any CUDA call, so these run without a GPU.
Pointers are fake values far apart, never dereferenced."""
import ctypes

import pytest

from block_quantized_matmul_gguf_gb300 import build, qmm

M = 1 << 24
OK, NULL, SHAPE = qmm.QMM_OK, qmm.QMM_ERR_NULL, qmm.QMM_ERR_SHAPE
ALIGN, UNSUPPORTED = qmm.QMM_ERR_ALIGN, qmm.QMM_ERR_UNSUPPORTED
FAR = 1 << 44
BIG = 1 << 40  # bytes of a workspace that is never too small


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return qmm.load()


def ref(s):
    return ctypes.addressof(s)


def test_packed_structs_are_the_compilers():
    for packer, struct in ((qmm._ROPE_ARGS, qmm.RopeArgs), (qmm._ROUTE_ARGS, qmm.RouteArgs),
                           (qmm._EXPERT_PLAN, qmm.ExpertPlan)):
        assert len(packer.pack(*(0 for _ in struct._fields_))) <= ctypes.sizeof(struct)
        # each field lies where the other layout has it
        for i, (name, kind) in enumerate(struct._fields_):
            values = [0] * len(struct._fields_)
            values[i] = 1
            raw = packer.pack(*values).ljust(ctypes.sizeof(struct), b"\0")
            assert getattr(struct.from_buffer_copy(raw), name) == 1


def cache(**kw):
    f = dict(k_codes=1 * M, k_scales=2 * M, v_codes=3 * M, v_scales=4 * M, num_pages=8, page_size=16,
             kv_heads=2, head_dim=64)
    f.update(kw)
    return qmm.KvQ4_0(**f)


def rope(**kw):
    f = dict(q=5 * M, q_stride=256, q_out=6 * M, q_out_stride=256, heads=4, k=7 * M, k_stride=128, v=8 * M,
             v_stride=128, type=0, slots=9 * M, positions=10 * M, n=4, table=11 * M, table_rows=32, rot=64,
             interleaved=0)
    f.update(kw)
    return qmm.RopeArgs(**f)


@pytest.mark.parametrize("kw,status", [
    (dict(n=0), OK), (dict(n=0, k=None, q_out=None), OK),
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(slots=None), NULL), (dict(positions=None), NULL),
    (dict(table=None), NULL), (dict(q_out=None), NULL),
    (dict(n=-1), SHAPE), (dict(type=2), SHAPE), (dict(rot=0), SHAPE), (dict(rot=63), SHAPE), (dict(rot=66), SHAPE),
    (dict(table_rows=0), SHAPE), (dict(k_stride=127), SHAPE), (dict(v_stride=64), SHAPE), (dict(q_stride=255), SHAPE),
    (dict(q_out_stride=255), SHAPE), (dict(heads=0), SHAPE),
    (dict(n=(1 << 30) + 1), UNSUPPORTED), (dict(table_rows=1 << 31), UNSUPPORTED),
    (dict(k_stride=1 << 31), UNSUPPORTED), (dict(heads=1025, q_stride=1025 * 64, q_out_stride=1025 * 64), UNSUPPORTED),
    (dict(k=7 * M + 2), ALIGN), (dict(type=1, k=7 * M + 1), ALIGN), (dict(q=5 * M + 1), ALIGN),
    (dict(q_out=6 * M + 2), ALIGN), (dict(slots=9 * M + 4), ALIGN), (dict(positions=10 * M + 2), ALIGN),
    (dict(table=11 * M + 1), ALIGN),
    (dict(q_out=5 * M), UNSUPPORTED), (dict(q_out=7 * M + 64), UNSUPPORTED), (dict(q_out=11 * M), UNSUPPORTED),
    (dict(k=1 * M), UNSUPPORTED), (dict(table=3 * M), UNSUPPORTED), (dict(q_out=2 * M), UNSUPPORTED),
])
def test_rotation_checks(lib, kw, status):
    assert lib.qmm_kv_append_rope_q4_0(ref(cache()), ref(rope(**kw)), None) == status


def test_rotation_needs_a_cache_and_arguments(lib):
    assert lib.qmm_kv_append_rope_q4_0(None, ref(rope()), None) == NULL
    assert lib.qmm_kv_append_rope_q4_0(ref(cache()), None, None) == NULL
    assert lib.qmm_kv_append_rope_q4_0(ref(cache(head_dim=96)), ref(rope()), None) == UNSUPPORTED


def route(**kw):
    f = dict(logits=1 * M, logits_stride=64, type=0, bias=2 * M, count=3 * M, tokens=600, experts=64, topk=8, score=0,
             groups=1, group_topk=1, group_best=1, renormalize=1, scale=1.0, ids=4 * M, weights=5 * M,
             expert_start=6 * M, pairs=7 * M, workspace=FAR, workspace_bytes=BIG)
    f.update(kw)
    return qmm.RouteArgs(**f)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=0), OK), (dict(tokens=0, logits=None), OK),
    (dict(tokens=-1), SHAPE), (dict(experts=0), SHAPE), (dict(topk=0), SHAPE), (dict(topk=65), SHAPE),
    (dict(type=2), SHAPE), (dict(score=2), SHAPE), (dict(score=-1), SHAPE), (dict(groups=0), SHAPE),
    (dict(groups=5), SHAPE), (dict(groups=8, group_topk=9), SHAPE), (dict(groups=8, group_topk=0), SHAPE),
    (dict(groups=16, group_topk=1), SHAPE), (dict(groups=8, group_topk=2, group_best=3), SHAPE),
    (dict(group_best=0), SHAPE), (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE),
    (dict(logits_stride=63), SHAPE),
    (dict(experts=1025, logits_stride=1025), UNSUPPORTED), (dict(topk=33), UNSUPPORTED),
    (dict(groups=64, group_topk=8), UNSUPPORTED), (dict(tokens=(1 << 27) + 1), UNSUPPORTED),
    (dict(logits_stride=1 << 31), UNSUPPORTED),
    (dict(logits=None), NULL), (dict(ids=None), NULL), (dict(weights=None), NULL), (dict(expert_start=None), NULL),
    (dict(pairs=None), NULL), (dict(workspace=None), NULL),
    (dict(logits=M + 2), ALIGN), (dict(type=1, logits=M + 1), ALIGN), (dict(bias=2 * M + 2), ALIGN),
    (dict(count=3 * M + 1), ALIGN), (dict(ids=4 * M + 2), ALIGN), (dict(weights=5 * M + 2), ALIGN),
    (dict(expert_start=6 * M + 1), ALIGN), (dict(pairs=7 * M + 3), ALIGN), (dict(workspace=FAR + 8), ALIGN),
    (dict(ids=1 * M), UNSUPPORTED), (dict(weights=4 * M + 64), UNSUPPORTED), (dict(pairs=2 * M), UNSUPPORTED),
    (dict(expert_start=3 * M), UNSUPPORTED), (dict(workspace=M), UNSUPPORTED),
])
def test_routing_checks(lib, kw, status):
    assert lib.qmm_route(ref(route(**kw)), None) == status


def test_routing_needs_arguments_and_room(lib):
    assert lib.qmm_route(None, None) == NULL
    need = lib.qmm_route_workspace_bytes(600, 64)
    assert need > 0
    assert lib.qmm_route(ref(route(workspace_bytes=need - 1)), None) == SHAPE
    assert lib.qmm_route_workspace_bytes(0, 64) == 0 == lib.qmm_route_workspace_bytes(4, 1025)
    sizes = [lib.qmm_route_workspace_bytes(t, 64) for t in (1, 128, 600, 5000, 1 << 20)]
    assert sizes == sorted(sizes)


def plan(**kw):
    f = dict(tokens=40, topk=2, experts=8, expert_start=1 * M, pairs=2 * M)
    f.update(kw)
    return qmm.ExpertPlan(**f)


def geglu(lib, p=None, wg=3 * M, wu=4 * M, x=5 * M, xs=256, xt=1, h=6 * M, hs=64, ht=1, n=64, k=256, ws=FAR, wsb=BIG, **kw):
    p = plan(**kw) if p is None else p
    return lib.qmm_experts_geglu_q4_0(p and ref(p), wg, wu, x, xs, xt, h, hs, ht, n, k, ws, wsb, None)


def down(lib, p=None, wd=3 * M, h=4 * M, hs=256, ht=1, ids=5 * M, weights=6 * M, y=7 * M, ys=64, yt=1, n=64, k=256,
         ws=FAR, wsb=BIG, **kw):
    p = plan(**kw) if p is None else p
    return lib.qmm_experts_down_q4_0(p and ref(p), wd, h, hs, ht, ids, weights, y, ys, yt, n, k, ws, wsb, None)


BOTH = [
    (dict(tokens=0), OK), (dict(tokens=0, expert_start=None, pairs=None), OK), (dict(tokens=-1), SHAPE),
    (dict(topk=0), SHAPE), (dict(experts=0), SHAPE), (dict(n=0), SHAPE), (dict(k=0), SHAPE), (dict(k=48), SHAPE),
    (dict(experts=1025), UNSUPPORTED), (dict(topk=33), UNSUPPORTED), (dict(tokens=1 << 30), UNSUPPORTED),
    (dict(n=(1 << 24) + 1), UNSUPPORTED), (dict(k=(1 << 20) + 32), UNSUPPORTED),
    (dict(expert_start=None), NULL), (dict(pairs=None), NULL),
    (dict(expert_start=M + 2), ALIGN), (dict(pairs=2 * M + 1), ALIGN),
]


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(wg=None), NULL), (dict(wu=None), NULL), (dict(x=None), NULL), (dict(h=None), NULL),
    (dict(xt=2), SHAPE), (dict(ht=-1), SHAPE), (dict(xs=255), SHAPE), (dict(hs=63), SHAPE),
    (dict(xs=1 << 31), UNSUPPORTED), (dict(hs=1 << 31), UNSUPPORTED),
    (dict(wg=3 * M + 8), ALIGN), (dict(wu=4 * M + 2), ALIGN), (dict(x=5 * M + 1), ALIGN), (dict(ht=0, h=6 * M + 2), ALIGN),
    (dict(ws=FAR + 8), ALIGN), (dict(wsb=16), SHAPE),
    (dict(h=5 * M + 64), UNSUPPORTED), (dict(h=3 * M), UNSUPPORTED), (dict(h=1 * M), UNSUPPORTED),
    (dict(ws=5 * M), UNSUPPORTED), (dict(ws=6 * M), UNSUPPORTED),
])
def test_geglu_checks(lib, kw, status):
    assert geglu(lib, **kw) == status


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(wd=None), NULL), (dict(h=None), NULL), (dict(y=None), NULL), (dict(ids=None), NULL),
    (dict(weights=None), NULL), (dict(ws=None), NULL),
    (dict(ht=2), SHAPE), (dict(yt=-1), SHAPE), (dict(hs=255), SHAPE), (dict(ys=63), SHAPE),
    (dict(hs=1 << 31), UNSUPPORTED), (dict(ys=1 << 31), UNSUPPORTED),
    (dict(wd=3 * M + 8), ALIGN), (dict(h=4 * M + 1), ALIGN), (dict(yt=0, y=7 * M + 2), ALIGN), (dict(ids=5 * M + 2), ALIGN),
    (dict(weights=6 * M + 1), ALIGN), (dict(ws=FAR + 4), ALIGN), (dict(wsb=16), SHAPE),
    (dict(y=4 * M + 64), UNSUPPORTED), (dict(y=5 * M), UNSUPPORTED), (dict(y=2 * M), UNSUPPORTED),
    (dict(ws=7 * M), UNSUPPORTED), (dict(ws=6 * M), UNSUPPORTED),
])
def test_down_checks(lib, kw, status):
    assert down(lib, **kw) == status


def test_products_need_a_plan(lib):
    assert lib.qmm_experts_geglu_q4_0(None, 3 * M, 4 * M, 5 * M, 256, 1, 6 * M, 64, 1, 64, 256, FAR, BIG, None) == NULL
    assert lib.qmm_experts_down_q4_0(None, 3 * M, 4 * M, 256, 1, 5 * M, 6 * M, 7 * M, 64, 1, 64, 256, FAR, BIG, None) == NULL


def test_workspace_sizes(lib):
    small, many = lib.qmm_experts_geglu_workspace_bytes, lib.qmm_experts_down_workspace_bytes
    assert small(1, 3, 8, 256) == 0  # few pairs for the experts: no rows to lay out
    assert small(2, 2, 8, 256) >= 4 * 256 * 2 and small(1, 1, 8, 4096) >= 4096 * 2
    assert small(2, 2, 8, 288) >= 4 * 512 * 2  # rows are laid out in multiples of 256
    assert small(0, 2, 8, 256) == small(4, 33, 8, 256) == small(4, 2, 1025, 256) == small(4, 2, 8, 1 << 21) == 0
    # z as fp32, or as bf16 with the rows of h behind it
    assert many(4, 2, 64, 256) >= 8 * 64 * 4 and many(4, 2, 64, 256) >= 8 * (64 + 256) * 2
    assert many(0, 2, 64, 256) == many(4, 0, 64, 256) == many(4, 2, 0, 256) == 0
    # 64-bit sizes
    assert many(1 << 20, 8, 8192, 2048) > 1 << 37
