"""Page plan, Q4_0 cache append and read on the GPU against plain references."""
import numpy as np
import pytest

import serving_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qmm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_quantized_matmul_gguf_gb300 import build, qmm as q
    build.build_library()
    q.load()
    q.qmm_get_device_error()
    return q


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def run_plan(qmm, cached, added, free, table, page, capacity):
    t = dev(table, torch.int32)
    out = dict(q_start=torch.full((len(cached) + 1,), -9, dtype=torch.int32).cuda(),
               kv_len=torch.full((len(cached),), -9, dtype=torch.int32).cuda(),
               slots=torch.full((capacity,), -9, dtype=torch.int64).cuda(),
               positions=torch.full((capacity,), -9, dtype=torch.int32).cuda(),
               taken=torch.full((1,), -9, dtype=torch.int32).cuda())
    qmm.qmm_kv_plan(dev(cached, torch.int32), dev(added, torch.int32), dev(free, torch.int32), t, page, **out)
    return [t.cpu().numpy()] + [out[k].cpu().numpy() for k in ("q_start", "kv_len", "slots", "positions", "taken")]


def same_plan(got, want):
    for g, w, name in zip(got, want, ("table", "q_start", "kv_len", "slots", "positions", "taken")):
        assert np.array_equal(g, w), name


def random_plan(rng, batch, page, top, more, spare=0):
    cached = rng.integers(0, top + 1, batch)
    added = rng.integers(0, more + 1, batch)
    width = max(1, int((-(-(cached + added) // page)).max()) + spare)
    had = -(-cached // page)
    ids = rng.permutation(int((-(-(cached + added) // page)).sum()) + 7)
    table = np.full((batch, width), -1)
    at = 0
    for b in range(batch):
        table[b, :had[b]] = ids[at:at + had[b]]
        at += had[b]
    return cached, added, ids[at:], table


@pytest.mark.parametrize("batch,page,top,more,pad", [
    (1, 16, 0, 1, 0), (1, 64, 100, 0, 3), (2, 16, 40, 1, 0), (16, 64, 4000, 1, 5), (33, 32, 70, 65, 1),
    (255, 16, 17, 33, 0), (257, 1024, 3000, 2, 9), (1000, 16, 50, 20, 100), (4099, 128, 300, 3, 1),
    (16384, 16, 20, 2, 0),
])
def test_plan(qmm, batch, page, top, more, pad):
    rng = np.random.default_rng(batch * 7 + page)
    cached, added, free, table = random_plan(rng, batch, page, top, more, spare=2)
    cap = int(added.sum()) + pad
    want = ref.plan(cached, added, free, table, page, cap)
    for _ in range(2):  # the same call again gives the same result
        same_plan(run_plan(qmm, cached, added, free, table, page, cap), want)
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


def test_plan_boundaries(qmm):
    """Lengths that end exactly at a page, start one, or add nothing."""
    cached = np.array([0, 16, 15, 17, 32, 0, 1])
    added = np.array([16, 1, 1, 0, 16, 0, 31])
    free = np.arange(100, 120)
    table = np.full((7, 4), -1)
    table[1, 0], table[2, 0], table[3, :2], table[4, :2], table[6, 0] = 3, 4, (5, 6), (7, 8), 9
    cap = int(added.sum())
    same_plan(run_plan(qmm, cached, added, free, table, 16, cap), ref.plan(cached, added, free, table, 16, cap))
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


def test_plan_shortages_are_marked_and_recorded(qmm):
    cached, added = np.array([16, 0, 5]), np.array([20, 40, 3])
    table = np.full((3, 2), -1)
    table[0, 0], table[2, 0] = 11, 12
    # the free list ends after two pages, and the table after two columns
    got = run_plan(qmm, cached, added, np.array([1, 2]), table, 16, 70)
    assert qmm.qmm_get_device_error() == qmm.QMM_ERR_INDEX
    want = ref.plan(cached, added, np.array([1, 2]), table, 16, 70)
    same_plan(got, want)
    assert (got[3][:63] < 0).any() and got[5][0] == 5
    # too little room for the tokens: q_start stops there
    got = run_plan(qmm, cached, added, np.arange(9), np.full((3, 9), 3), 16, 30)
    assert qmm.qmm_get_device_error() == qmm.QMM_ERR_INDEX
    assert got[1].tolist() == [0, 20, 30, 30]
    # a negative length counts as none
    got = run_plan(qmm, np.array([-5, 3]), np.array([2, -1]), np.arange(9), np.full((2, 3), 3), 16, 4)
    assert qmm.qmm_get_device_error() == qmm.QMM_ERR_INDEX
    assert got[1].tolist() == [0, 2, 2] and got[2].tolist() == [2, 3]
    # no free pages at all, no capacity at all
    e = torch.empty(0, dtype=torch.int32).cuda()
    out = [torch.zeros(n, dtype=torch.int32).cuda() for n in (2, 1)]
    taken = torch.zeros(1, dtype=torch.int32).cuda()
    qmm.qmm_kv_plan(dev([16], torch.int32), dev([0], torch.int32), e, dev([[4]], torch.int32), 16, out[0], out[1],
                    torch.empty(0, dtype=torch.int64).cuda(), e, taken)
    assert qmm.qmm_get_device_error() == qmm.QMM_OK
    assert out[0].tolist() == [0, 0] and out[1].tolist() == [16] and taken.item() == 0


def cache_arrays(cache):
    return [t.cpu().numpy() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,page,n,dtype", [(1, 16, 1, "f32"), (2, 64, 16, "f32"), (3, 32, 77, "bf16"),
                                                (4, 128, 1000, "f32"), (8, 1024, 33, "bf16")])
def test_append_then_read(qmm, dim, heads, page, n, dtype):
    g = torch.Generator().manual_seed(dim + n)
    pages = -(-n // page) + 3
    k, v = (torch.randn(n, heads, dim, generator=g) * torch.exp(2 * torch.randn(n, heads, 1, generator=g))
            for _ in range(2))
    k[0, 0, :32] = 0.0                      # an empty block
    v[0, 0, :32] = torch.arange(32) - 15.5  # +-15.5: the positive one is the extreme
    v[0, 0, 31] = 15.5
    v[0, 0, 0] = -15.5
    if dtype == "bf16":
        k, v = k.bfloat16(), v.bfloat16()
    slots = torch.randperm(pages * page, generator=g)[:n]
    cache = qmm.kv_cache_q4_0(pages, page, heads, dim)
    qmm.qmm_kv_append_q4_0(cache, k.cuda(), v.cuda(), slots.cuda())
    kc, ks, vc, vs = cache_arrays(cache)
    at, off = slots.numpy() // page, slots.numpy() % page
    for x, codes, scales in ((k, kc, ks), (v, vc, vs)):
        wc, ws = ref.quantize(x.float().numpy())
        # the definition in fp32: the division is the one rounding before round()
        b = x.float().numpy().reshape(n, heads, -1, 32)
        f = ws.astype(np.float32)[..., None]
        r = np.divide(b, f, out=np.zeros_like(b), where=f != 0)
        c = np.where(f == 0, 8, np.clip(np.rint(r) + 8, 0, 15)).astype(np.uint8)
        c = (c[..., :16] | (c[..., 16:] << 4)).reshape(wc.shape)
        assert np.array_equal(scales[at, :, off], ws)
        assert np.array_equal(codes[at, :, off], c)
        untouched = np.ones((pages, page), bool)
        untouched[at, off] = False
        assert not codes.transpose(0, 2, 1, 3)[untouched].any()
        assert not scales.transpose(0, 2, 1, 3)[untouched].view(np.uint16).any()
    out = [torch.full((n, heads, dim), 7.0).cuda() for _ in range(2)]
    qmm.qmm_kv_read_q4_0(cache, slots.cuda(), *out)
    for y, codes, scales in zip(out, (kc, vc), (ks, vs)):
        want = ref.values(codes[at, :, off], scales[at, :, off])
        assert np.array_equal(y.cpu().numpy(), want.astype(np.float32))
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


def test_append_extreme_values(qmm):
    """Non-finite blocks read back as NaN, huge ones saturate the scale, tiny
    ones underflow to zero; their neighbours are not affected."""
    x = torch.zeros(6, 1, 64)
    x[:, :, 32:] = torch.linspace(-3, 4, 32)
    x[0, 0, 5] = float("nan")
    x[1, 0, 6] = float("inf")
    x[2, 0, 31] = -float("inf")
    x[3, 0, :32] = 3.0e38
    x[4, 0, :32] = -1.0e-9
    x[5, 0, :32] = torch.linspace(-1e-6, 2e-6, 32)  # a subnormal scale
    cache = qmm.kv_cache_q4_0(1, 16, 1, 64)
    slots = torch.arange(6).cuda()
    qmm.qmm_kv_append_q4_0(cache, x.cuda(), x.cuda(), slots)
    y, z = torch.empty(6, 1, 64).cuda(), torch.empty(6, 1, 64).cuda()
    qmm.qmm_kv_read_q4_0(cache, slots, y, z)
    y = y.cpu().numpy()[:, 0]
    assert np.array_equal(y, z.cpu().numpy()[:, 0], equal_nan=True)
    assert np.isnan(y[:3, :32]).all()
    assert (y[3, :32] == 8 * 65504.0).all()
    assert (y[4, :32] == 0).all()
    c, s = ref.quantize(x.numpy()[:, 0])
    want = ref.values(c, s)
    assert np.array_equal(y[5], want[5].astype(np.float32))
    assert np.array_equal(y[:, 32:], want[:, 32:].astype(np.float32))


@pytest.mark.parametrize("offset,dtype", [(0, torch.float32), (1, torch.float32), (2, torch.bfloat16),
                                          (3, torch.bfloat16)])
def test_append_strided_and_unaligned_rows(qmm, offset, dtype):
    n, heads, dim, wide = 9, 2, 128, 2 * 256 + 7
    host = torch.randn(n * wide + 8).to(dtype)
    base = host.cuda()
    rows = base[offset:offset + n * wide].view(n, wide)
    k, v = rows[:, :256].view(n, heads, dim), rows[:, 256:512].view(n, heads, dim)
    slots = torch.arange(n).flip(0).cuda()
    a, b = (qmm.kv_cache_q4_0(1, 16, heads, dim) for _ in range(2))
    qmm.qmm_kv_append_q4_0(a, k, v, slots)
    dense = host[offset:offset + n * wide].view(n, wide)
    qmm.qmm_kv_append_q4_0(b, dense[:, :256].reshape(n, heads, dim).cuda(),
                           dense[:, 256:512].reshape(n, heads, dim).cuda(), slots)
    for x, y in zip(cache_arrays(a), cache_arrays(b)):
        assert np.array_equal(x, y) and x.any()
    out = torch.empty(n * 256 + 1).cuda()
    y = torch.empty(n, heads, dim).cuda()
    qmm.qmm_kv_read_q4_0(a, slots, out[1:].view(n, heads, dim), None)  # 4-byte aligned only
    qmm.qmm_kv_read_q4_0(a, slots, y, None)
    assert torch.equal(out.cpu()[1:].view(n, heads, dim), y.cpu())


def test_slots_outside_the_cache_are_skipped(qmm):
    cache = qmm.kv_cache_q4_0(2, 16, 1, 64)
    x = torch.ones(4, 1, 64).cuda()
    qmm.qmm_kv_append_q4_0(cache, x, x, torch.tensor([-1, 3, -1, 31]).cuda())
    assert qmm.qmm_get_device_error() == qmm.QMM_OK
    y = torch.full((3, 1, 64), 5.0).cuda()
    qmm.qmm_kv_read_q4_0(cache, torch.tensor([3, -1, 31]).cuda(), y, None)
    assert y[0].eq(1).all() and y[1].eq(0).all() and y[2].eq(1).all()
    assert qmm.qmm_get_device_error() == qmm.QMM_OK
    before = cache_arrays(cache)
    for bad in (32, -2, 1 << 40):
        qmm.qmm_kv_append_q4_0(cache, x[:1], x[:1], torch.tensor([bad]).cuda())
        assert qmm.qmm_get_device_error() == qmm.QMM_ERR_INDEX
        qmm.qmm_kv_read_q4_0(cache, torch.tensor([bad]).cuda(), y[:1], None)
        assert qmm.qmm_get_device_error() == qmm.QMM_ERR_INDEX
        assert y[0].eq(0).all()
    for a, b in zip(before, cache_arrays(cache)):
        assert np.array_equal(a, b)


def test_append_past_32_bit_offsets(qmm):
    """Slots whose codes lie beyond 4 GiB of the array."""
    pages, page, heads, dim = 18000, 1024, 2, 256
    cache = qmm.KvCacheQ4_0(*(torch.empty((pages, heads, page, w), dtype=t, device="cuda")
                              for w, t in ((128, torch.uint8), (8, torch.float16)) * 2))
    x = torch.randn(5, heads, dim).cuda()
    slots = torch.tensor([pages * page - 1, 0, 17500 * page + 5, 16384 * page, 16383 * page + 1023]).cuda()
    qmm.qmm_kv_append_q4_0(cache, x, x + 1, slots)
    k, v = torch.empty_like(x), torch.empty_like(x)
    qmm.qmm_kv_read_q4_0(cache, slots, k, v)
    for y, z in ((k, x), (v, x + 1)):
        c, s = ref.quantize(z.cpu().numpy())
        assert np.abs(y.cpu().numpy() - ref.values(c, s)).max() < 1e-6
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


def test_python_refusals(qmm):
    cache = qmm.kv_cache_q4_0(1, 16, 2, 64)
    x, s = torch.zeros(3, 2, 64).cuda(), torch.zeros(3, dtype=torch.int64).cuda()
    for k, v, slots in ((x.half(), x.half(), s), (x, x.bfloat16(), s), (x[:2], x, s), (x, x, s.int()),
                        (x[:, :, :32], x, s), (x.cpu(), x, s), (x.transpose(1, 2), x, s)):
        with pytest.raises(ValueError):
            qmm.qmm_kv_append_q4_0(cache, k, v, slots)
    with pytest.raises(ValueError):
        qmm.qmm_kv_read_q4_0(cache, s, torch.zeros(2, 2, 64).cuda(), None)
    with pytest.raises(ValueError):
        qmm.KvCacheQ4_0(cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales[:, :, :8])
    with pytest.raises(qmm.QmmError):
        bad = qmm.kv_cache_q4_0(1, 16, 2, 96)
        qmm.qmm_kv_read_q4_0(bad, s, torch.zeros(3, 2, 96).cuda(), None)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_append_quotients_near_halves(qmm, dtype):
    """Values at halves of the scale and a few units in the last place beside
    them round as the fp32 quotient does, ties to even."""
    rng = np.random.default_rng(12)
    n, dim = 512, 256
    d = np.abs(rng.standard_normal((n, 1, dim // 32, 1))).astype(np.float16).astype(np.float32)
    x = (rng.integers(-8, 8, (n, 1, dim // 32, 32)) + 0.5).astype(np.float32) * d
    x = (x.view(np.int32) + rng.integers(-3, 4, x.shape, dtype=np.int32)).view(np.float32)
    x = np.clip(x, -8 * d, 8 * d)
    x[..., 3] = (-8 * d)[..., 0]  # the extreme: the scale is d
    t = torch.from_numpy(x.reshape(n, 1, dim))
    t = t.bfloat16() if dtype == "bf16" else t
    b = t.float().numpy().reshape(n, 1, -1, 32)
    cache = qmm.kv_cache_q4_0(n // 64, 64, 1, dim)
    qmm.qmm_kv_append_q4_0(cache, t.cuda(), t.cuda(), torch.arange(n).cuda())
    kc, ks, vc, vs = (a.reshape(n, 1, -1) for a in cache_arrays(cache))
    f = ks.astype(np.float32).reshape(n, 1, -1, 1)
    assert np.array_equal(ks, vs) and np.array_equal(kc, vc)
    assert np.array_equal(ks, ref.quantize(t.float().numpy())[1])
    c = np.clip(np.rint(b / f) + 8, 0, 15).astype(np.uint8)
    assert np.array_equal(kc, (c[..., :16] | (c[..., 16:] << 4)).reshape(kc.shape))
