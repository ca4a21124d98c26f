"""A workspace for some number of tokens serves any smaller number."""
import pytest

from block_quantized_matmul_gguf_gb300 import build, qmm


@pytest.fixture(scope="module")
def lib():
    try:
        build.build_library()
    except RuntimeError as e:
        pytest.skip(str(e))
    return qmm.load()


@pytest.mark.parametrize("experts", [1, 64, 256, 1024])
def test_sizes_never_fall(lib, experts):
    counts = sorted({n + d for n in (1, 128, 256, 512, 1024, 8192, 10000, 16384, 32768, 49152, 1 << 20, 1 << 30) for d in (-1, 0, 1)
                     if 0 < n + d <= 1 << 30})
    sizes = [lib.qmm_route_workspace_bytes(n, experts) for n in counts]
    assert sizes == sorted(sizes)
    assert lib.qmm_route_workspace_bytes(512, experts) == 0 < lib.qmm_route_workspace_bytes(513, experts)


@pytest.mark.gpu
@pytest.mark.parametrize("most,tokens", [(10000, 8191), (16385, 8192), (8193, 8192), (16385, 16384), (600, 512), (40000, 700)])
def test_a_larger_workspace_serves(most, tokens):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build_library()
    experts, topk = 32, 4
    logits = torch.randn(tokens, experts, generator=torch.Generator().manual_seed(tokens)).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    out = [[torch.empty(tokens, topk, **i32), torch.empty(tokens, topk, device="cuda"), torch.empty(experts + 1, **i32),
            torch.empty(tokens * topk, **i32)] for _ in range(2)]
    qmm.qmm_route(logits, *out[0])
    qmm.qmm_route(logits, *out[1], workspace=qmm.route_workspace(most, experts))
    assert all(torch.equal(a, b) for a, b in zip(*out))
    ids = out[1][0].reshape(-1)
    assert torch.equal(out[1][3].long(), ids.sort(stable=True).indices)
    assert qmm.qmm_get_device_error() == qmm.QMM_OK
