"""The append with the rotation: codes and scales bit for bit against fp32
products and sums rounded once, queries against the same."""
import numpy as np
import pytest

import experts_ref
import serving_ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qmm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_quantized_matmul_gguf_gb300 import build, qmm
    build.build_library()
    return qmm


def arrays(cache):
    return [t.cpu().numpy() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]


def expected(cache, k, v, slots, positions, table, rot, interleaved):
    """The four arrays of a cache of zeros after the append."""
    want = [np.zeros_like(a) for a in arrays(cache)]
    kk = experts_ref.turn(k, table, positions, rot, interleaved)
    for half, x in ((0, kk), (2, np.asarray(v, dtype=np.float32))):
        codes, scales = serving_ref.quantize(x)
        for i, (s, p) in enumerate(zip(slots, positions)):
            if s >= 0 and p >= 0:
                want[half][s // cache.page_size, :, s % cache.page_size] = codes[i]
                want[half + 1][s // cache.page_size, :, s % cache.page_size] = scales[i]
    return want


def same(got, want):
    for g, w in zip(got, want):
        assert np.array_equal(g.view(np.uint16) if g.dtype == np.float16 else g,
                              w.view(np.uint16) if w.dtype == np.float16 else w)


def rounded(x, dtype):
    return torch.from_numpy(x).to(dtype).float().numpy()


@pytest.mark.parametrize("n,heads,kv,dim,rot", [(1, 1, 1, 64, 64), (3, 4, 2, 64, 40), (16, 8, 2, 256, 256), (77, 6, 3, 128, 64),
                                                (130, 16, 4, 128, 2), (700, 8, 4, 256, 232), (5, 32, 8, 128, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_keys_values_and_queries(qmm, n, heads, kv, dim, rot, interleaved, dtype):
    g = torch.Generator().manual_seed(n * 31 + rot)
    both = torch.randn(n, heads + 2 * kv, dim, generator=g).to(dtype).cuda()
    q, k, v = both[:, :heads], both[:, heads:heads + kv], both[:, heads + kv:]  # columns of one projection
    far = 5000
    table = qmm.rope_table(far, rot)
    positions = torch.randint(0, far, (n,), generator=g, dtype=torch.int32)
    pages = -(-n // 16) + 2
    slots = torch.randperm(pages * 16, generator=g)[:n]
    cache = qmm.kv_cache_q4_0(pages, 16, kv, dim)
    q_out = torch.full((n, heads, dim), 7.0, dtype=dtype, device="cuda")
    qmm.qmm_kv_append_rope_q4_0(cache, k, v, slots.cuda(), positions.cuda(), table, q=q, q_out=q_out, interleaved=interleaved)
    t, at = table.cpu().numpy(), positions.numpy()
    same(arrays(cache), expected(cache, k.float().cpu().numpy(), v.float().cpu().numpy(), slots.numpy(), at, t, rot, interleaved))
    want = rounded(experts_ref.turn(q.float().cpu().numpy(), t, at, rot, interleaved), dtype)
    assert np.array_equal(q_out.float().cpu().numpy(), want)
    assert qmm.qmm_get_device_error() == qmm.QMM_OK
    # without queries the cache is the same
    other = qmm.kv_cache_q4_0(pages, 16, kv, dim)
    qmm.qmm_kv_append_rope_q4_0(other, k, v, slots.cuda(), positions.cuda(), table, interleaved=interleaved)
    same(arrays(other), arrays(cache))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("off", [1, 2])
def test_rows_and_tables_without_alignment(qmm, interleaved, off):
    n, heads, kv, dim, rot = 40, 2, 2, 64, 64
    g = torch.Generator().manual_seed(5)
    flat = torch.randn(n, (heads + 2 * kv) * dim + 7, generator=g).bfloat16().cuda()
    part = flat[:, off:off + (heads + 2 * kv) * dim].unflatten(1, (-1, dim))
    q, k, v = part[:, :heads], part[:, heads:heads + kv], part[:, heads + kv:]
    room = torch.empty(100 * rot + 3, device="cuda")
    table = room[off:off + 100 * rot].view(100, rot)
    table.copy_(qmm.rope_table(100, rot, base=500000.0))
    positions = torch.arange(n, dtype=torch.int32) * 2
    slots = torch.arange(n)
    cache = qmm.kv_cache_q4_0(3, 16, kv, dim)
    q_out = torch.empty(n, heads, dim, dtype=torch.bfloat16, device="cuda")
    qmm.qmm_kv_append_rope_q4_0(cache, k, v, slots.cuda(), positions.cuda(), table, q=q, q_out=q_out, interleaved=interleaved)
    t = table.cpu().numpy()
    same(arrays(cache), expected(cache, k.float().cpu().numpy(), v.float().cpu().numpy(), slots.numpy(), positions.numpy(), t,
                                 rot, interleaved))
    want = experts_ref.turn(q.float().cpu().numpy(), t, positions.numpy(), rot, interleaved)
    assert np.array_equal(q_out.float().cpu().numpy(), rounded(want, torch.bfloat16))


def test_position_zero_is_the_plain_append(qmm):
    n, kv, dim = 50, 2, 128
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(n, kv, dim, generator=g).cuda() for _ in range(2))
    slots = torch.arange(n).cuda()
    a, b = qmm.kv_cache_q4_0(4, 16, kv, dim), qmm.kv_cache_q4_0(4, 16, kv, dim)
    qmm.qmm_kv_append_q4_0(a, k, v, slots)
    qmm.qmm_kv_append_rope_q4_0(b, k, v, slots, torch.zeros(n, dtype=torch.int32).cuda(), qmm.rope_table(1, dim))
    same(arrays(a), arrays(b))


def test_tokens_left_out(qmm):
    """Padding, tokens without a slot, and indices outside their arrays."""
    n, heads, kv, dim = 6, 2, 1, 64
    g = torch.Generator().manual_seed(9)
    q, k, v = (torch.randn(n, h, dim, generator=g).cuda() for h in (heads, kv, kv))
    table = qmm.rope_table(10, dim)
    slots = torch.tensor([3, -1, -1, 5, 40, 7]).cuda()
    positions = torch.tensor([9, 4, -1, -1, 2, 1], dtype=torch.int32).cuda()
    cache = qmm.kv_cache_q4_0(2, 16, kv, dim)
    q_out = torch.full((n, heads, dim), 7.0, device="cuda")
    qmm.qmm_kv_append_rope_q4_0(cache, k, v, slots, positions, table, q=q, q_out=q_out)
    assert qmm.qmm_get_device_error() == qmm.QMM_ERR_INDEX  # slot 40
    want_slots, want_pos = [3, -1, -1, -1, -1, 7], [9, 4, -1, -1, 2, 1]  # its query is rotated
    same(arrays(cache), expected(cache, k.cpu().numpy(), v.cpu().numpy(), want_slots, want_pos, table.cpu().numpy(), dim, False))
    want = experts_ref.turn(q.cpu().numpy(), table.cpu().numpy(), want_pos, dim, False)
    for i, p in enumerate(want_pos):
        assert np.array_equal(q_out[i].cpu().numpy(), want[i] if p >= 0 else np.full((heads, dim), 7.0, np.float32))
    for bad in (10, -2):
        positions.fill_(3)
        positions[0] = bad
        slots = torch.arange(n).cuda()
        q_out.fill_(7.0)
        qmm.qmm_kv_append_rope_q4_0(cache, k, v, slots, positions, table, q=q, q_out=q_out)
        assert qmm.qmm_get_device_error() == qmm.QMM_ERR_INDEX
        assert (q_out[0] == 7.0).all() and (q_out[1:] != 7.0).all()


def test_values_that_are_no_numbers(qmm):
    k = torch.ones(3, 1, 64).cuda()
    v = torch.ones(3, 1, 64).cuda()
    k[0, 0, 1], k[1, 0, 40], v[2, 0, 3] = float("nan"), float("inf"), float("-inf")
    cache = qmm.kv_cache_q4_0(1, 16, 1, 64)
    slots = torch.arange(3).cuda()
    qmm.qmm_kv_append_rope_q4_0(cache, k, v, slots, torch.tensor([1, 2, 3], dtype=torch.int32).cuda(), qmm.rope_table(4, 64))
    back = [torch.empty(3, 1, 64, device="cuda") for _ in range(2)]
    qmm.qmm_kv_read_q4_0(cache, slots, *back)
    bad = [torch.isnan(b).view(3, 2, 32).all(-1).cpu().tolist() for b in back]
    assert bad[0] == [[True, True], [True, True], [False, False]]  # both of the pair's blocks
    assert bad[1] == [[False, False], [False, False], [True, False]]


def test_streams_graphs_and_refusals(qmm):
    n, kv, dim = 9, 2, 64
    g = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn(n, kv, dim, generator=g).cuda() for _ in range(3))
    table = qmm.rope_table(64, dim)
    slots, positions = torch.arange(n).cuda(), torch.arange(n, dtype=torch.int32).cuda()
    cache = qmm.kv_cache_q4_0(1, 16, kv, dim)
    q_out = torch.empty_like(q)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        qmm.qmm_kv_append_rope_q4_0(cache, k, v, slots, positions, table, q=q, q_out=q_out)
    positions.add_(50)
    k.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    same(arrays(cache), expected(cache, k.cpu().numpy(), v.cpu().numpy(), range(n), range(50, 50 + n), table.cpu().numpy(), dim,
                                 False))
    for kw in (dict(q=q), dict(q=q, q_out=q_out.bfloat16()), dict(q=q[:, :1], q_out=q_out)):
        with pytest.raises(ValueError):
            qmm.qmm_kv_append_rope_q4_0(cache, k, v, slots, positions, table, **kw)
    with pytest.raises(ValueError):
        qmm.qmm_kv_append_rope_q4_0(cache, k, v, slots, positions[:3], table)
    with pytest.raises(qmm.QmmError):  # in place
        qmm.qmm_kv_append_rope_q4_0(cache, k, v, slots, positions, table, q=q, q_out=q)
    with pytest.raises(qmm.QmmError):  # more than the head
        qmm.qmm_kv_append_rope_q4_0(cache, k, v, slots, positions, qmm.rope_table(64, 128))
