// qmm_api.cu -- the C ABI (include/qmm.h): argument checks, per-device state
// (error word, SM count), launches.  No entry point allocates device memory.
#include "../../include/qmm.h"
#include "qmm_internal.h"

#include <cudaTypedefs.h>

#include <atomic>
#include <mutex>

namespace qmm {

// Device error word: written by kernels that give up a bounded wait, read
// and cleared by qmm_get_device_error().  One per GPU (module-scope device
// variable; no allocation).
__device__ uint32_t g_device_error = 0;

namespace {

constexpr uint64_t kDefaultTimeoutNs = 2000000000ull;

std::atomic<uint64_t> g_timeout_ns{kDefaultTimeoutNs};

struct DeviceState {
    std::once_flag once;
    cudaError_t init_err = cudaSuccess;
    uint32_t *err_word = nullptr;
    int sms = 0;
};
DeviceState g_dev[kMaxDevices];

// Per-device set-up, once, with that device current.
DeviceState *device_state(cudaError_t *err) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        *err = e != cudaSuccess ? e : cudaErrorInvalidDevice;
        return nullptr;
    }
    DeviceState &st = g_dev[dev];
    std::call_once(st.once, [&st, dev]() {
        void *p = nullptr;
        st.init_err = cudaGetSymbolAddress(&p, g_device_error);
        if (st.init_err == cudaSuccess) {
            st.err_word = static_cast<uint32_t *>(p);
            st.init_err = cudaDeviceGetAttribute(&st.sms, cudaDevAttrMultiProcessorCount, dev);
        }
    });
    *err = st.init_err;
    return st.init_err == cudaSuccess ? &st : nullptr;
}

bool make_ctx(LaunchCtx *ctx) {
    cudaError_t e;
    DeviceState *st = device_state(&e);
    if (!st) return false;
    ctx->err = st->err_word;
    ctx->timeout_ns = g_timeout_ns.load(std::memory_order_relaxed);
    return true;
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

qmm_status from_cuda(cudaError_t e) { return e == cudaSuccess ? QMM_OK : QMM_ERR_CUDA; }

qmm_status check_wk(const void *w, int64_t n, int64_t k) {
    if (!w) return QMM_ERR_NULL;
    if (n < 1 || k < kQK || k % kQK != 0) return QMM_ERR_SHAPE;
    // byte offsets of the largest index must fit comfortably in 64 bits
    if (n > (int64_t(1) << 40) || k > (int64_t(1) << 31)) return QMM_ERR_SHAPE;
    return QMM_OK;
}

// [a, a+an) and [b, b+bn) overlap
bool overlaps(const void *a, size_t an, const void *b, size_t bn) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + bn && y < x + an;
}

qmm_status dequant(Fmt fmt, const void *w, float *out, int64_t n, int64_t k,
                   qmm_stream_t stream) {
    qmm_status s = check_wk(w, n, k);
    if (s != QMM_OK) return s;
    if (!out) return QMM_ERR_NULL;
    if (!aligned(out, 4)) return QMM_ERR_ALIGN;
    LaunchCtx ctx;
    if (!make_ctx(&ctx)) return QMM_ERR_CUDA;
    return from_cuda(launch_dequant(fmt, static_cast<const uint8_t *>(w), out, n, k,
                                    reinterpret_cast<cudaStream_t>(stream), ctx));
}

qmm_status gemv(Fmt fmt, const qmm_gemv_out *outs, int count, const float *x, int m, int64_t k,
                qmm_stream_t stream) {
    if (!outs || !x) return QMM_ERR_NULL;
    if (count < 1 || count > QMM_GEMV_MAX_OUTPUTS) return QMM_ERR_SHAPE;
    if (m < 1 || m > QMM_GEMV_MAX_M) return QMM_ERR_SHAPE;
    if (!aligned(x, 4)) return QMM_ERR_ALIGN;
    GemvProblem probs[QMM_GEMV_MAX_OUTPUTS];
    for (int i = 0; i < count; ++i) {
        const qmm_status s = check_wk(outs[i].w, outs[i].n, k);
        if (s != QMM_OK) return s;
        if (!outs[i].y) return QMM_ERR_NULL;
        if (!aligned(outs[i].y, 4)) return QMM_ERR_ALIGN;
        probs[i] = GemvProblem{outs[i].w, outs[i].y, outs[i].n};
    }
    // no output may overlap an input or another output
    const size_t xbytes = sizeof(float) * static_cast<size_t>(m) * k;
    for (int i = 0; i < count; ++i) {
        const size_t ybytes = sizeof(float) * static_cast<size_t>(m) * outs[i].n;
        if (overlaps(outs[i].y, ybytes, x, xbytes)) return QMM_ERR_UNSUPPORTED;
        for (int j = 0; j < count; ++j) {
            const size_t wbytes = static_cast<size_t>(outs[j].n) * (k / kQK) * block_bytes(fmt);
            if (overlaps(outs[i].y, ybytes, outs[j].w, wbytes)) return QMM_ERR_UNSUPPORTED;
            if (j != i && overlaps(outs[i].y, ybytes, outs[j].y,
                                   sizeof(float) * static_cast<size_t>(m) * outs[j].n))
                return QMM_ERR_UNSUPPORTED;
        }
    }
    LaunchCtx ctx;
    if (!make_ctx(&ctx)) return QMM_ERR_CUDA;
    return from_cuda(launch_gemv(fmt, probs, count, x, m, k,
                                 reinterpret_cast<cudaStream_t>(stream), ctx));
}

// Memory a kernel on the current device may read and write at address p:
// that device's memory, managed memory, or page-locked host memory mapped
// at its host address.  Pageable host memory is refused (a kernel access
// to it would fault).
bool device_accessible(const void *p) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    cudaPointerAttributes a;
    if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
        (void)cudaGetLastError();  // the failed query is not a launch error: clear it
        return false;
    }
    switch (a.type) {
    case cudaMemoryTypeDevice:
        return a.device == dev;
    case cudaMemoryTypeManaged:
        return true;
    case cudaMemoryTypeHost:
        return a.devicePointer == p;
    default:
        return false;
    }
}

qmm_status check_workspace(const void *ws, size_t ws_bytes, size_t need) {
    if (!aligned(ws, 16)) return QMM_ERR_ALIGN;
    if (ws_bytes < need) return QMM_ERR_SHAPE;
    return QMM_OK;
}

// Checks shared by the tensor-core GEMM entry points (plain product): y is
// fp32 [m][n], written with 4-byte stores; y may overlap neither input.
qmm_status check_gemm(Fmt fmt, const void *w, const uint16_t *x_bf16, const float *y, int64_t m,
                      int64_t n, int64_t k) {
    qmm_status s = check_wk(w, n, k);
    if (s != QMM_OK) return s;
    if (!x_bf16 || !y) return QMM_ERR_NULL;
    if (m < 1) return QMM_ERR_SHAPE;
    if (k % 256 != 0 || m > kGemmMaxM || n > kGemmMaxN || k > kGemmMaxK)
        return QMM_ERR_UNSUPPORTED;
    if (!aligned(w, 16) || !aligned(x_bf16, 16) || !aligned(y, 4)) return QMM_ERR_ALIGN;
    const size_t ybytes = sizeof(float) * static_cast<size_t>(m) * n;
    const size_t wbytes = static_cast<size_t>(n) * (k / kQK) * block_bytes(fmt);
    if (overlaps(y, ybytes, w, wbytes) || overlaps(y, ybytes, x_bf16, 2 * static_cast<size_t>(m) * k))
        return QMM_ERR_UNSUPPORTED;
    return QMM_OK;
}

qmm_status gemm(Fmt fmt, const void *w, const uint16_t *x_bf16, float *y, int64_t m, int64_t n,
                int64_t k, qmm_stream_t stream, void *ws = nullptr, size_t ws_bytes = 0) {
    qmm_status s = check_gemm(fmt, w, x_bf16, y, m, n, k);
    if (s != QMM_OK) return s;
    const bool two_phase = ws != nullptr && use_two_phase_gemm(m, n, k);
    const size_t wbytes = static_cast<size_t>(n) * (k / kQK) * block_bytes(fmt);
    const size_t ybytes = sizeof(float) * static_cast<size_t>(m) * n;
    if (ws != nullptr) {
        // two phases: the dequantised weights; one phase (short prompts):
        // room for K-split partial products
        const size_t need = gemm_workspace_bytes(n, k, false);
        s = check_workspace(ws, ws_bytes, need);
        if (s != QMM_OK) return s;
        if (overlaps(ws, need, w, wbytes) || overlaps(ws, need, x_bf16, 2 * static_cast<size_t>(m) * k) ||
            overlaps(ws, need, y, ybytes))
            return QMM_ERR_UNSUPPORTED;
    }
    LaunchCtx ctx;
    if (!make_ctx(&ctx)) return QMM_ERR_CUDA;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const uint8_t *wb = static_cast<const uint8_t *>(w);
    if (two_phase)
        return from_cuda(launch_gemm_two_phase(fmt, wb, x_bf16, y, m, n, k,
                                               static_cast<uint16_t *>(ws), st, ctx));
    // K-split budget: fixed by the shape (not by what this caller happens to
    // give), so that every workspace and the prefill entry's scratch choose
    // the same split and give the same bits
    float *part = static_cast<float *>(ws);
    const size_t budget = ws != nullptr ? fused_part_budget(n, k) : 0;
    return from_cuda(fmt == Fmt::Q4_0 ? launch_gemm_q4_0(wb, x_bf16, y, m, n, k, st, ctx, part, budget)
                                      : launch_gemm_q8_0(wb, x_bf16, y, m, n, k, st, ctx, part, budget));
}

// ---- serving operators ----------------------------------------------------------

constexpr int64_t kMaxRows = int64_t(1) << 30;  // tokens of one call
constexpr int64_t kMaxIndex = (int64_t(1) << 31) - 1;

// log2 of a page size the cache takes (a power of two, 16..1024), else -1.
int page_shift_of(int page_size) {
    for (int s = 4; s <= 10; ++s)
        if (page_size == 1 << s) return s;
    return -1;
}

size_t codes_bytes(const KvCache &c) {
    return (static_cast<size_t>(c.num_pages) * c.kv_heads << c.page_shift) * (c.head_dim / 2);
}
size_t scales_bytes(const KvCache &c) {
    return (static_cast<size_t>(c.num_pages) * c.kv_heads << c.page_shift) * (c.head_dim / kQK) * 2;
}

// Sizes that define a cache; pointers are check_cache's part.
qmm_status check_cache_sizes(const qmm_kv_q4_0 *cache, KvCache *c) {
    if (!cache) return QMM_ERR_NULL;
    if (cache->num_pages < 1 || cache->kv_heads < 1 || cache->head_dim < 1 || cache->page_size < 1)
        return QMM_ERR_SHAPE;
    const int shift = page_shift_of(cache->page_size);
    if (shift < 0 || (cache->head_dim != 64 && cache->head_dim != 128 && cache->head_dim != 256))
        return QMM_ERR_UNSUPPORTED;
    if (cache->num_pages > kMaxIndex || cache->kv_heads > 1024 ||
        (cache->num_pages * cache->kv_heads) << shift > kMaxIndex)
        return QMM_ERR_UNSUPPORTED;
    *c = KvCache{cache->k_codes, cache->k_scales, cache->v_codes, cache->v_scales,
                 cache->num_pages, shift, cache->kv_heads, cache->head_dim};
    return QMM_OK;
}

qmm_status check_cache(const qmm_kv_q4_0 *cache, KvCache *c) {
    const qmm_status s = check_cache_sizes(cache, c);
    if (s != QMM_OK) return s;
    if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales) return QMM_ERR_NULL;
    if (!aligned(c->k_codes, 16) || !aligned(c->k_scales, 16) || !aligned(c->v_codes, 16) ||
        !aligned(c->v_scales, 16))
        return QMM_ERR_ALIGN;
    return QMM_OK;
}

bool overlaps_cache(const KvCache &c, const void *p, size_t bytes) {
    return overlaps(p, bytes, c.k_codes, codes_bytes(c)) || overlaps(p, bytes, c.v_codes, codes_bytes(c)) ||
           overlaps(p, bytes, c.k_scales, scales_bytes(c)) || overlaps(p, bytes, c.v_scales, scales_bytes(c));
}

bool valid_dtype(qmm_dtype t) { return t == QMM_F32 || t == QMM_BF16; }
size_t dtype_bytes(qmm_dtype t) { return t == QMM_F32 ? 4 : 2; }

// Bytes from the first to the last element of `rows` rows `stride` elements apart.
size_t rows_bytes(int64_t rows, int64_t stride, int64_t width, size_t size) {
    return rows < 1 ? 0 : (static_cast<size_t>(rows - 1) * stride + width) * size;
}

struct Range {
    const void *p;
    size_t bytes;
};

// No output range may overlap an input or another output (null ranges are absent).
bool outputs_clear(const Range *outs, int no, const Range *ins, int ni) {
    for (int i = 0; i < no; ++i) {
        if (!outs[i].p || !outs[i].bytes) continue;
        for (int j = 0; j < ni; ++j)
            if (ins[j].p && ins[j].bytes && overlaps(outs[i].p, outs[i].bytes, ins[j].p, ins[j].bytes))
                return false;
        for (int j = 0; j < i; ++j)
            if (outs[j].p && outs[j].bytes && overlaps(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes))
                return false;
    }
    return true;
}

}  // namespace

bool encode_tmap_2d(CUtensorMap *map, CUtensorMapDataType dtype, const void *base,
                    uint64_t inner, uint64_t outer, uint64_t outer_stride_bytes,
                    uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swizzle) {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, []() {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    if (!fn) return false;
    const cuuint64_t dims[2] = {inner, outer};
    const cuuint64_t strides[1] = {outer_stride_bytes};
    const cuuint32_t box[2] = {box_inner, box_outer};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, dtype, 2, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int current_device() {
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess ? dev : 0;
}

int device_sm_count() {
    cudaError_t e;
    DeviceState *st = device_state(&e);
    return st ? st->sms : 1;
}

// ---- self-test: a wait that nothing completes ---------------------------------
__global__ void selftest_wait_kernel(LaunchCtx ctx) {
    __shared__ __align__(8) uint64_t bar;
    if (threadIdx.x == 0) mbar_init(&bar, 1);
    fence_mbar_init();
    __syncthreads();
    if (threadIdx.x == 0) mbar_wait(&bar, 0, ctx);  // never completes: bounded by ctx.timeout_ns
    __syncthreads();
}

cudaError_t launch_selftest_wait(cudaStream_t stream, const LaunchCtx &ctx) {
    return launch_kernel(selftest_wait_kernel, dim3(1), dim3(32), 0, stream, 1, ctx);
}

}  // namespace qmm

using namespace qmm;

extern "C" {

qmm_status qmm_dequant_q4_0(const void *w, float *out, int64_t n, int64_t k,
                            qmm_stream_t stream) {
    return dequant(Fmt::Q4_0, w, out, n, k, stream);
}

qmm_status qmm_dequant_q8_0(const void *w, float *out, int64_t n, int64_t k,
                            qmm_stream_t stream) {
    return dequant(Fmt::Q8_0, w, out, n, k, stream);
}

qmm_status qmm_copy(void *dst, const void *src, size_t bytes, qmm_stream_t stream) {
    if (bytes == 0) return QMM_OK;
    if (!dst || !src) return QMM_ERR_NULL;
    if (overlaps(dst, bytes, src, bytes)) return QMM_ERR_UNSUPPORTED;
    if (!device_accessible(src) || !device_accessible(dst)) return QMM_ERR_UNSUPPORTED;
    cudaError_t e;
    if (!device_state(&e)) return QMM_ERR_CUDA;  // the SM count for the grid
    return from_cuda(launch_copy(dst, src, bytes, reinterpret_cast<cudaStream_t>(stream)));
}

qmm_status qmm_gemv_q4_0(const void *w, const float *x, float *y, int m, int64_t n, int64_t k,
                         qmm_stream_t stream) {
    const qmm_gemv_out one = {w, y, n};
    return gemv(Fmt::Q4_0, &one, 1, x, m, k, stream);
}

qmm_status qmm_gemv_q8_0(const void *w, const float *x, float *y, int m, int64_t n, int64_t k,
                         qmm_stream_t stream) {
    const qmm_gemv_out one = {w, y, n};
    return gemv(Fmt::Q8_0, &one, 1, x, m, k, stream);
}

qmm_status qmm_gemv_q4_0_multi(const qmm_gemv_out *outs, int count, const float *x, int m,
                               int64_t k, qmm_stream_t stream) {
    return gemv(Fmt::Q4_0, outs, count, x, m, k, stream);
}

qmm_status qmm_gemv_q8_0_multi(const qmm_gemv_out *outs, int count, const float *x, int m,
                               int64_t k, qmm_stream_t stream) {
    return gemv(Fmt::Q8_0, outs, count, x, m, k, stream);
}

qmm_status qmm_gemv_q4_0_geglu(const void *wg, const void *wu, const float *x, float *h, int m,
                               int64_t n, int64_t k, qmm_stream_t stream) {
    qmm_status s = check_wk(wg, n, k);
    if (s == QMM_OK) s = check_wk(wu, n, k);
    if (s != QMM_OK) return s;
    if (!x || !h) return QMM_ERR_NULL;
    if (m < 1 || m > QMM_GEMV_MAX_M) return QMM_ERR_SHAPE;
    if (!aligned(x, 4) || !aligned(h, 4)) return QMM_ERR_ALIGN;
    const size_t hbytes = sizeof(float) * static_cast<size_t>(m) * n;
    const size_t wbytes = static_cast<size_t>(n) * (k / kQK) * kQ4_0Bytes;
    if (overlaps(h, hbytes, x, sizeof(float) * static_cast<size_t>(m) * k) ||
        overlaps(h, hbytes, wg, wbytes) || overlaps(h, hbytes, wu, wbytes))
        return QMM_ERR_UNSUPPORTED;
    LaunchCtx ctx;
    if (!make_ctx(&ctx)) return QMM_ERR_CUDA;
    const GemvProblem gate_up[2] = {{wg, h, n}, {wu, nullptr, n}};
    return from_cuda(launch_geglu_q4_0(gate_up, x, m, k, reinterpret_cast<cudaStream_t>(stream), ctx));
}

qmm_status qmm_gemv_q4_0_tc(const void *w, const float *x, float *y, int m, int64_t n, int64_t k,
                            qmm_stream_t stream) {
    qmm_status s = check_wk(w, n, k);
    if (s != QMM_OK) return s;
    if (!x || !y) return QMM_ERR_NULL;
    if (m < 1 || m > QMM_GEMV_MAX_M) return QMM_ERR_SHAPE;
    if (!gemv_tc_shape_ok(m, n, k)) return QMM_ERR_UNSUPPORTED;
    if (!aligned(w, 16) || !aligned(x, 16) || !aligned(y, 4)) return QMM_ERR_ALIGN;
    const size_t ybytes = sizeof(float) * static_cast<size_t>(m) * n;
    const size_t wbytes = static_cast<size_t>(n) * (k / kQK) * kQ4_0Bytes;
    if (overlaps(y, ybytes, w, wbytes) || overlaps(y, ybytes, x, sizeof(float) * static_cast<size_t>(m) * k))
        return QMM_ERR_UNSUPPORTED;
    LaunchCtx ctx;
    if (!make_ctx(&ctx)) return QMM_ERR_CUDA;
    return from_cuda(launch_gemv_tc_q4_0(static_cast<const uint8_t *>(w), x, y, m, n, k,
                                         reinterpret_cast<cudaStream_t>(stream), ctx));
}

qmm_status qmm_gemm_q4_0(const void *w, const uint16_t *x_bf16, float *y, int64_t m, int64_t n,
                         int64_t k, qmm_stream_t stream) {
    return gemm(Fmt::Q4_0, w, x_bf16, y, m, n, k, stream);
}

qmm_status qmm_gemm_q8_0(const void *w, const uint16_t *x_bf16, float *y, int64_t m, int64_t n,
                         int64_t k, qmm_stream_t stream) {
    return gemm(Fmt::Q8_0, w, x_bf16, y, m, n, k, stream);
}

qmm_status qmm_gemm_q4_0_prefill(const void *w, const uint16_t *x_bf16, float *y, int64_t m,
                                 int64_t n, int64_t k, qmm_stream_t stream) {
    qmm_status s = check_gemm(Fmt::Q4_0, w, x_bf16, y, m, n, k);
    if (s != QMM_OK) return s;
    if (k > kPrefillMaxK) return QMM_ERR_SCRATCH;
    LaunchCtx ctx;
    if (!make_ctx(&ctx)) return QMM_ERR_CUDA;
    return from_cuda(launch_gemm_q4_0_prefill(static_cast<const uint8_t *>(w), x_bf16, y, m, n, k,
                                              reinterpret_cast<cudaStream_t>(stream), ctx));
}

size_t qmm_gemm_workspace_bytes(int64_t n, int64_t k) {
    if (n < 1 || k < 1) return 0;
    return gemm_workspace_bytes(n, k, false);
}

size_t qmm_gemm_geglu_workspace_bytes(int64_t n, int64_t k) {
    if (n < 1 || k < 1) return 0;
    return gemm_workspace_bytes(n, k, true);
}

qmm_status qmm_gemm_q4_0_ws(const void *w, const uint16_t *x_bf16, float *y, int64_t m, int64_t n,
                            int64_t k, void *workspace, size_t workspace_bytes,
                            qmm_stream_t stream) {
    return gemm(Fmt::Q4_0, w, x_bf16, y, m, n, k, stream, workspace, workspace_bytes);
}

qmm_status qmm_gemm_q8_0_ws(const void *w, const uint16_t *x_bf16, float *y, int64_t m, int64_t n,
                            int64_t k, void *workspace, size_t workspace_bytes,
                            qmm_stream_t stream) {
    return gemm(Fmt::Q8_0, w, x_bf16, y, m, n, k, stream, workspace, workspace_bytes);
}

qmm_status qmm_gemm_q4_0_geglu(const void *wg, const void *wu, const uint16_t *x_bf16,
                               uint16_t *h_bf16, int64_t m, int64_t n, int64_t k,
                               qmm_stream_t stream) {
    return qmm_gemm_q4_0_geglu_ws(wg, wu, x_bf16, h_bf16, m, n, k, nullptr, 0, stream);
}

qmm_status qmm_gemm_q4_0_geglu_ws(const void *wg, const void *wu, const uint16_t *x_bf16,
                                  uint16_t *h_bf16, int64_t m, int64_t n, int64_t k,
                                  void *workspace, size_t workspace_bytes, qmm_stream_t stream) {
    qmm_status s = check_wk(wg, n, k);
    if (s == QMM_OK) s = check_wk(wu, n, k);
    if (s != QMM_OK) return s;
    if (!x_bf16 || !h_bf16) return QMM_ERR_NULL;
    if (m < 1) return QMM_ERR_SHAPE;
    if (k % 256 != 0 || m > kGemmMaxM || n > kGemmMaxN || k > kGemmMaxK) return QMM_ERR_UNSUPPORTED;
    if (!aligned(wg, 16) || !aligned(wu, 16) || !aligned(x_bf16, 16) || !aligned(h_bf16, 2))
        return QMM_ERR_ALIGN;
    const size_t hbytes = sizeof(uint16_t) * static_cast<size_t>(m) * n;
    const size_t wbytes = static_cast<size_t>(n) * (k / kQK) * kQ4_0Bytes;
    if (overlaps(h_bf16, hbytes, x_bf16, sizeof(uint16_t) * static_cast<size_t>(m) * k) ||
        overlaps(h_bf16, hbytes, wg, wbytes) || overlaps(h_bf16, hbytes, wu, wbytes))
        return QMM_ERR_UNSUPPORTED;
    const bool two_phase = workspace != nullptr && use_two_phase_geglu(m, k);
    if (two_phase) {
        const size_t need = gemm_workspace_bytes(n, k, true);
        s = check_workspace(workspace, workspace_bytes, need);
        if (s != QMM_OK) return s;
        if (overlaps(workspace, need, wg, wbytes) || overlaps(workspace, need, wu, wbytes) ||
            overlaps(workspace, need, x_bf16, sizeof(uint16_t) * static_cast<size_t>(m) * k) ||
            overlaps(workspace, need, h_bf16, hbytes))
            return QMM_ERR_UNSUPPORTED;
    }
    LaunchCtx ctx;
    if (!make_ctx(&ctx)) return QMM_ERR_CUDA;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (two_phase)
        return from_cuda(launch_gemm_geglu_two_phase(static_cast<const uint8_t *>(wg),
                                                     static_cast<const uint8_t *>(wu), x_bf16,
                                                     h_bf16, m, n, k,
                                                     static_cast<uint16_t *>(workspace), st, ctx));
    return from_cuda(launch_gemm_q4_0_geglu(static_cast<const uint8_t *>(wg),
                                            static_cast<const uint8_t *>(wu), x_bf16, h_bf16, m, n,
                                            k, st, ctx));
}

qmm_status qmm_kv_plan(const int32_t *cached, const int32_t *added, int batch,
                       const int32_t *free_pages, int64_t num_free, int32_t *table,
                       int64_t table_width, int page_size, int32_t *q_start, int32_t *kv_len,
                       int64_t *slots, int32_t *positions, int64_t capacity, int32_t *taken,
                       qmm_stream_t stream) {
    if (!cached || !added || !table || !q_start || !kv_len || !taken) return QMM_ERR_NULL;
    if (batch < 1 || num_free < 0 || table_width < 1 || capacity < 0 || page_size < 1) return QMM_ERR_SHAPE;
    if ((num_free > 0 && !free_pages) || (capacity > 0 && (!slots || !positions))) return QMM_ERR_NULL;
    const int shift = page_shift_of(page_size);
    if (shift < 0 || batch > kMaxBatch || num_free > kMaxIndex || table_width > kMaxIndex ||
        capacity > kMaxIndex)
        return QMM_ERR_UNSUPPORTED;
    if (!aligned(cached, 4) || !aligned(added, 4) || !aligned(free_pages, 4) || !aligned(table, 4) ||
        !aligned(q_start, 4) || !aligned(kv_len, 4) || !aligned(slots, 8) || !aligned(positions, 4) ||
        !aligned(taken, 4))
        return QMM_ERR_ALIGN;
    const size_t b = static_cast<size_t>(batch), n = static_cast<size_t>(capacity);
    const Range ins[] = {{cached, 4 * b}, {added, 4 * b}, {free_pages, 4 * static_cast<size_t>(num_free)}};
    const Range outs[] = {{table, 4 * b * static_cast<size_t>(table_width)}, {q_start, 4 * (b + 1)},
                          {kv_len, 4 * b}, {slots, 8 * n}, {positions, 4 * n}, {taken, 4}};
    if (!outputs_clear(outs, 6, ins, 3)) return QMM_ERR_UNSUPPORTED;
    LaunchCtx ctx;
    if (!make_ctx(&ctx)) return QMM_ERR_CUDA;
    const KvPlan plan = {cached, added, free_pages, table, q_start, kv_len, positions, taken, slots,
                         num_free, table_width, capacity, batch, shift};
    return from_cuda(launch_kv_plan(plan, reinterpret_cast<cudaStream_t>(stream), ctx));
}

qmm_status qmm_kv_append_q4_0(const qmm_kv_q4_0 *cache, const void *k, int64_t k_stride, const void *v,
                              int64_t v_stride, qmm_dtype type, const int64_t *slots, int64_t n,
                              qmm_stream_t stream) {
    KvCache c;
    const qmm_status s = check_cache(cache, &c);
    if (s != QMM_OK) return s;
    if (n < 0 || !valid_dtype(type)) return QMM_ERR_SHAPE;
    if (n == 0) return QMM_OK;
    if (!k || !v || !slots) return QMM_ERR_NULL;
    const int64_t width = static_cast<int64_t>(c.kv_heads) * c.head_dim;
    if (k_stride < width || v_stride < width) return QMM_ERR_SHAPE;
    if (n > kMaxRows || k_stride > kMaxIndex || v_stride > kMaxIndex) return QMM_ERR_UNSUPPORTED;
    const size_t size = dtype_bytes(type);
    if (!aligned(k, size) || !aligned(v, size) || !aligned(slots, 8)) return QMM_ERR_ALIGN;
    if (overlaps_cache(c, k, rows_bytes(n, k_stride, width, size)) ||
        overlaps_cache(c, v, rows_bytes(n, v_stride, width, size)) ||
        overlaps_cache(c, slots, 8 * static_cast<size_t>(n)))
        return QMM_ERR_UNSUPPORTED;
    LaunchCtx ctx;
    if (!make_ctx(&ctx)) return QMM_ERR_CUDA;
    return from_cuda(launch_kv_append(c, k, k_stride, v, v_stride, type == QMM_BF16, slots, n,
                                      reinterpret_cast<cudaStream_t>(stream), ctx));
}

qmm_status qmm_kv_append_rope_q4_0(const qmm_kv_q4_0 *cache, const qmm_rope_args *args, qmm_stream_t stream) {
    KvCache c;
    const qmm_status s = check_cache(cache, &c);
    if (s != QMM_OK) return s;
    if (!args) return QMM_ERR_NULL;
    const qmm_rope_args &a = *args;
    if (a.n < 0 || !valid_dtype(a.type) || a.rot < 2 || a.rot % 2 != 0 || a.rot > c.head_dim || a.table_rows < 1)
        return QMM_ERR_SHAPE;
    if (a.n == 0) return QMM_OK;
    if (!a.k || !a.v || !a.slots || !a.positions || !a.table || (a.q && !a.q_out)) return QMM_ERR_NULL;
    const int64_t width = static_cast<int64_t>(c.kv_heads) * c.head_dim;
    const int64_t q_width = a.q ? static_cast<int64_t>(a.heads) * c.head_dim : 0;
    if (a.k_stride < width || a.v_stride < width) return QMM_ERR_SHAPE;
    if (a.q && (a.heads < 1 || a.q_stride < q_width || a.q_out_stride < q_width)) return QMM_ERR_SHAPE;
    if (a.n > kMaxRows || a.k_stride > kMaxIndex || a.v_stride > kMaxIndex || a.table_rows > kMaxIndex ||
        (a.q && (a.heads > 1024 || a.q_stride > kMaxIndex || a.q_out_stride > kMaxIndex)))
        return QMM_ERR_UNSUPPORTED;
    const size_t size = dtype_bytes(a.type);
    if (!aligned(a.k, size) || !aligned(a.v, size) || !aligned(a.slots, 8) || !aligned(a.positions, 4) ||
        !aligned(a.table, 4) || (a.q && (!aligned(a.q, size) || !aligned(a.q_out, size))))
        return QMM_ERR_ALIGN;
    const Range ins[] = {{a.q, rows_bytes(a.n, a.q_stride, q_width, size)},
                         {a.k, rows_bytes(a.n, a.k_stride, width, size)},
                         {a.v, rows_bytes(a.n, a.v_stride, width, size)},
                         {a.slots, 8 * static_cast<size_t>(a.n)}, {a.positions, 4 * static_cast<size_t>(a.n)},
                         {a.table, 4 * static_cast<size_t>(a.table_rows) * a.rot}};
    const Range out = {a.q ? a.q_out : nullptr, rows_bytes(a.n, a.q_out_stride, q_width, size)};
    if (!outputs_clear(&out, 1, ins, 6)) return QMM_ERR_UNSUPPORTED;
    for (const Range &r : ins)
        if (r.p && r.bytes && overlaps_cache(c, r.p, r.bytes)) return QMM_ERR_UNSUPPORTED;
    if (out.p && overlaps_cache(c, out.p, out.bytes)) return QMM_ERR_UNSUPPORTED;
    LaunchCtx ctx;
    if (!make_ctx(&ctx)) return QMM_ERR_CUDA;
    const RopeArgs r = {a.q, a.k, a.v, a.q ? a.q_out : nullptr, a.table, a.positions, a.slots, a.q ? a.q_stride : 0,
                        a.q ? a.q_out_stride : 0, a.k_stride, a.v_stride, a.table_rows, a.n, a.q ? a.heads : 0, a.rot,
                        a.interleaved != 0, a.type == QMM_BF16};
    return from_cuda(launch_kv_append_rope(c, r, reinterpret_cast<cudaStream_t>(stream), ctx));
}

qmm_status qmm_kv_read_q4_0(const qmm_kv_q4_0 *cache, const int64_t *slots, int64_t n, float *k_out,
                            float *v_out, qmm_stream_t stream) {
    KvCache c;
    const qmm_status s = check_cache(cache, &c);
    if (s != QMM_OK) return s;
    if (n < 0) return QMM_ERR_SHAPE;
    if (n == 0) return QMM_OK;
    if (!slots || (!k_out && !v_out)) return QMM_ERR_NULL;
    if (n > kMaxRows) return QMM_ERR_UNSUPPORTED;
    if (!aligned(slots, 8) || !aligned(k_out, 4) || !aligned(v_out, 4)) return QMM_ERR_ALIGN;
    const size_t bytes = 4 * static_cast<size_t>(n) * c.kv_heads * c.head_dim;
    const Range ins[] = {{slots, 8 * static_cast<size_t>(n)}};
    const Range outs[] = {{k_out, bytes}, {v_out, bytes}};
    if (!outputs_clear(outs, 2, ins, 1) || (k_out && overlaps_cache(c, k_out, bytes)) ||
        (v_out && overlaps_cache(c, v_out, bytes)))
        return QMM_ERR_UNSUPPORTED;
    LaunchCtx ctx;
    if (!make_ctx(&ctx)) return QMM_ERR_CUDA;
    return from_cuda(launch_kv_read(c, slots, n, k_out, v_out, reinterpret_cast<cudaStream_t>(stream), ctx));
}

size_t qmm_attn_q4_0_workspace_bytes(const qmm_kv_q4_0 *cache, int heads) {
    KvCache c;
    if (check_cache_sizes(cache, &c) != QMM_OK || heads < 1 || heads % c.kv_heads != 0) return 0;
    return attn_workspace_bytes(c, heads);
}

qmm_status qmm_attn_q4_0(const qmm_kv_q4_0 *cache, const qmm_attn_args *args, qmm_stream_t stream) {
    KvCache c;
    qmm_status s = check_cache(cache, &c);
    if (s != QMM_OK) return s;
    if (!args) return QMM_ERR_NULL;
    const qmm_attn_args &a = *args;
    if (a.batch < 1 || a.total_q < 0 || a.max_q < 1 || a.heads < 1 || a.heads % c.kv_heads != 0 ||
        a.table_width < 1 || a.window < 0 || (a.window > 0 && !a.causal) || !(a.scale - a.scale == 0.0f) ||
        !valid_dtype(a.q_type) || !valid_dtype(a.out_type))
        return QMM_ERR_SHAPE;
    if (a.total_q == 0) return QMM_OK;
    if (!a.q || !a.out || !a.table || !a.q_start || !a.kv_len) return QMM_ERR_NULL;
    const int64_t width = static_cast<int64_t>(a.heads) * c.head_dim;
    if (a.q_stride < width || a.out_stride < width) return QMM_ERR_SHAPE;
    if (a.batch > kMaxBatch || a.total_q > kMaxRows || a.heads > 1024 || a.table_width > kMaxIndex ||
        a.q_stride > kMaxIndex || a.out_stride > kMaxIndex)
        return QMM_ERR_UNSUPPORTED;
    if (!aligned(a.q, dtype_bytes(a.q_type)) || !aligned(a.out, dtype_bytes(a.out_type)) ||
        !aligned(a.lse, 4) || !aligned(a.table, 4) || !aligned(a.q_start, 4) || !aligned(a.kv_len, 4))
        return QMM_ERR_ALIGN;
    const size_t need = attn_workspace_bytes(c, a.heads);
    if (need) {
        if (!a.workspace) return QMM_ERR_NULL;
        s = check_workspace(a.workspace, a.workspace_bytes, need);
        if (s != QMM_OK) return s;
    }
    const size_t out_bytes = rows_bytes(a.total_q, a.out_stride, width, dtype_bytes(a.out_type));
    const size_t lse_bytes = 4 * static_cast<size_t>(a.total_q) * a.heads, b = static_cast<size_t>(a.batch);
    const Range ins[] = {{a.q, rows_bytes(a.total_q, a.q_stride, width, dtype_bytes(a.q_type))},
                         {a.table, 4 * b * static_cast<size_t>(a.table_width)},
                         {a.q_start, 4 * (b + 1)}, {a.kv_len, 4 * b}};
    const Range outs[] = {{a.out, out_bytes}, {a.lse, lse_bytes}, {a.workspace, need}};
    if (!outputs_clear(outs, 3, ins, 4)) return QMM_ERR_UNSUPPORTED;
    for (const Range &o : outs)
        if (o.p && o.bytes && overlaps_cache(c, o.p, o.bytes)) return QMM_ERR_UNSUPPORTED;
    LaunchCtx ctx;
    if (!make_ctx(&ctx)) return QMM_ERR_CUDA;
    const AttnArgs k = {a.q, a.out, a.lse, a.table, a.q_start, a.kv_len, a.q_stride, a.out_stride,
                        a.table_width, a.total_q, a.batch, a.max_q, a.heads, a.causal != 0, a.window,
                        a.scale, a.q_type == QMM_BF16, a.out_type == QMM_BF16, a.workspace};
    return from_cuda(launch_attn(c, k, reinterpret_cast<cudaStream_t>(stream), ctx));
}

size_t qmm_route_workspace_bytes(int64_t tokens, int experts) {
    if (tokens < 1 || experts < 1 || tokens > kMaxRows || experts > kMaxExperts) return 0;
    return route_workspace_bytes(tokens, experts);
}

qmm_status qmm_route(const qmm_route_args *args, qmm_stream_t stream) {
    if (!args) return QMM_ERR_NULL;
    const qmm_route_args &a = *args;
    if (a.tokens < 0 || a.experts < 1 || a.topk < 1 || a.groups < 1 || a.group_topk < 1 || a.group_topk > a.groups ||
        (a.group_best != 1 && a.group_best != 2) || !valid_dtype(a.type) || !(a.scale - a.scale == 0.0f) ||
        (a.score != QMM_SCORE_SOFTMAX && a.score != QMM_SCORE_SIGMOID))
        return QMM_ERR_SHAPE;
    if (a.experts % a.groups != 0 || a.topk > a.experts / a.groups * a.group_topk || a.logits_stride < a.experts)
        return QMM_ERR_SHAPE;
    if (a.experts > kMaxExperts || a.topk > kMaxTopk || a.groups > kMaxGroups || a.tokens > kMaxRows / a.topk ||
        a.logits_stride > kMaxIndex)
        return QMM_ERR_UNSUPPORTED;
    if (a.tokens == 0) return QMM_OK;
    if (!a.logits || !a.ids || !a.weights || !a.expert_start || !a.pairs) return QMM_ERR_NULL;
    if (!aligned(a.logits, dtype_bytes(a.type)) || !aligned(a.bias, 4) || !aligned(a.count, 4) || !aligned(a.ids, 4) ||
        !aligned(a.weights, 4) || !aligned(a.expert_start, 4) || !aligned(a.pairs, 4))
        return QMM_ERR_ALIGN;
    const size_t need = route_workspace_bytes(a.tokens, a.experts);
    if (need) {
        if (!a.workspace) return QMM_ERR_NULL;
        const qmm_status s = check_workspace(a.workspace, a.workspace_bytes, need);
        if (s != QMM_OK) return s;
    }
    const size_t e = static_cast<size_t>(a.experts), list = 4 * static_cast<size_t>(a.tokens) * a.topk;
    const Range ins[] = {{a.logits, rows_bytes(a.tokens, a.logits_stride, a.experts, dtype_bytes(a.type))},
                         {a.bias, 4 * e}, {a.count, 4}};
    const Range outs[] = {{a.ids, list}, {a.weights, list}, {a.expert_start, 4 * (e + 1)}, {a.pairs, list},
                          {a.workspace, need}};
    if (!outputs_clear(outs, 5, ins, 3)) return QMM_ERR_UNSUPPORTED;
    LaunchCtx ctx;
    if (!make_ctx(&ctx)) return QMM_ERR_CUDA;
    const RouteArgs r = {a.logits, a.bias, a.count, a.ids, a.weights, a.expert_start, a.pairs, a.workspace,
                         a.logits_stride, a.tokens, a.experts, a.topk, a.groups, a.group_topk, a.group_best,
                         static_cast<int>(a.score), a.scale, a.type == QMM_BF16, a.renormalize != 0};
    return from_cuda(launch_route(r, reinterpret_cast<cudaStream_t>(stream), ctx));
}

namespace {

constexpr int64_t kExpertsMaxN = int64_t(1) << 24, kExpertsMaxK = int64_t(1) << 20;

// Checks shared by the experts' products.  `w`: weights of one kind.
qmm_status check_experts(const qmm_expert_plan *plan, const void *w, int64_t n, int64_t k, ExpertsPlan *out) {
    if (!plan) return QMM_ERR_NULL;
    if (plan->tokens < 0 || plan->topk < 1 || plan->experts < 1) return QMM_ERR_SHAPE;
    if (n < 1 || k < kQK || k % kQK != 0) return QMM_ERR_SHAPE;
    if (plan->experts > kMaxExperts || plan->topk > kMaxTopk || plan->tokens > kMaxRows / plan->topk || n > kExpertsMaxN ||
        k > kExpertsMaxK)
        return QMM_ERR_UNSUPPORTED;
    *out = ExpertsPlan{plan->expert_start, plan->pairs, plan->tokens * plan->topk, plan->experts, plan->topk};
    if (plan->tokens == 0) return QMM_OK;
    if (!w || !plan->expert_start || !plan->pairs) return QMM_ERR_NULL;
    if (!aligned(w, 16) || !aligned(plan->expert_start, 4) || !aligned(plan->pairs, 4)) return QMM_ERR_ALIGN;
    return QMM_OK;
}

size_t experts_bytes(const ExpertsPlan &p, int64_t n, int64_t k) {
    return static_cast<size_t>(p.experts) * n * (k / kQK) * kQ4_0Bytes;
}

}  // namespace

size_t qmm_experts_geglu_workspace_bytes(int64_t tokens, int topk, int experts, int64_t k) {
    if (tokens < 1 || topk < 1 || topk > kMaxTopk || experts < 1 || experts > kMaxExperts || tokens > kMaxRows / topk ||
        k < kQK || k > kExpertsMaxK || !experts_take_room(tokens * topk, experts, k))
        return 0;
    return experts_rows_bytes(tokens * topk, k);
}

qmm_status qmm_experts_geglu_q4_0(const qmm_expert_plan *plan, const void *wg, const void *wu, const void *x, int64_t x_stride,
                                  qmm_dtype x_type, void *h, int64_t h_stride, qmm_dtype h_type, int64_t n, int64_t k,
                                  void *workspace, size_t workspace_bytes, qmm_stream_t stream) {
    ExpertsPlan p;
    qmm_status s = check_experts(plan, wg, n, k, &p);
    if (s == QMM_OK) s = check_experts(plan, wu, n, k, &p);
    if (s != QMM_OK) return s;
    if (!valid_dtype(x_type) || !valid_dtype(h_type) || x_stride < k || h_stride < n) return QMM_ERR_SHAPE;
    if (x_stride > kMaxIndex || h_stride > kMaxIndex) return QMM_ERR_UNSUPPORTED;
    if (p.pairs_total == 0) return QMM_OK;
    if (!x || !h) return QMM_ERR_NULL;
    if (!aligned(x, dtype_bytes(x_type)) || !aligned(h, dtype_bytes(h_type))) return QMM_ERR_ALIGN;
    const size_t need = workspace ? qmm_experts_geglu_workspace_bytes(plan->tokens, p.topk, p.experts, k) : 0;
    if (need) {
        s = check_workspace(workspace, workspace_bytes, need);
        if (s != QMM_OK) return s;
    }
    const size_t wbytes = experts_bytes(p, n, k);
    const Range ins[] = {{wg, wbytes}, {wu, wbytes}, {x, rows_bytes(plan->tokens, x_stride, k, dtype_bytes(x_type))},
                         {p.expert_start, 4 * (static_cast<size_t>(p.experts) + 1)},
                         {p.pairs, 4 * static_cast<size_t>(p.pairs_total)}};
    const Range outs[] = {{h, rows_bytes(p.pairs_total, h_stride, n, dtype_bytes(h_type))}, {workspace, need}};
    if (!outputs_clear(outs, 2, ins, 5)) return QMM_ERR_UNSUPPORTED;
    LaunchCtx ctx;
    if (!make_ctx(&ctx)) return QMM_ERR_CUDA;
    const ExpertsGeglu a = {p, static_cast<const uint8_t *>(wg), static_cast<const uint8_t *>(wu), x, h, need ? workspace : nullptr,
                            x_stride, h_stride, n, k, x_type == QMM_BF16, h_type == QMM_BF16};
    return from_cuda(launch_experts_geglu(a, reinterpret_cast<cudaStream_t>(stream), ctx));
}

size_t qmm_experts_down_workspace_bytes(int64_t tokens, int topk, int64_t n, int64_t k) {
    if (tokens < 1 || topk < 1 || topk > kMaxTopk || tokens > kMaxRows / topk || n < 1 || n > kExpertsMaxN || k < kQK ||
        k > kExpertsMaxK)
        return 0;
    return experts_down_workspace_bytes(tokens * topk, n, k);
}

qmm_status qmm_experts_down_q4_0(const qmm_expert_plan *plan, const void *wd, const void *h, int64_t h_stride, qmm_dtype h_type,
                                 const int32_t *ids, const float *weights, void *y, int64_t y_stride, qmm_dtype y_type,
                                 int64_t n, int64_t k, void *workspace, size_t workspace_bytes, qmm_stream_t stream) {
    ExpertsPlan p;
    qmm_status s = check_experts(plan, wd, n, k, &p);
    if (s != QMM_OK) return s;
    if (!valid_dtype(h_type) || !valid_dtype(y_type) || h_stride < k || y_stride < n) return QMM_ERR_SHAPE;
    if (h_stride > kMaxIndex || y_stride > kMaxIndex) return QMM_ERR_UNSUPPORTED;
    if (p.pairs_total == 0) return QMM_OK;
    if (!h || !ids || !weights || !y || !workspace) return QMM_ERR_NULL;
    if (!aligned(h, dtype_bytes(h_type)) || !aligned(y, dtype_bytes(y_type)) || !aligned(ids, 4) || !aligned(weights, 4))
        return QMM_ERR_ALIGN;
    const size_t need = experts_down_workspace_bytes(p.pairs_total, n, k);
    s = check_workspace(workspace, workspace_bytes, need);
    if (s != QMM_OK) return s;
    const size_t list = 4 * static_cast<size_t>(p.pairs_total);
    const Range ins[] = {{wd, experts_bytes(p, n, k)}, {h, rows_bytes(p.pairs_total, h_stride, k, dtype_bytes(h_type))},
                         {p.expert_start, 4 * (static_cast<size_t>(p.experts) + 1)}, {p.pairs, list}, {ids, list},
                         {weights, list}};
    const Range outs[] = {{y, rows_bytes(plan->tokens, y_stride, n, dtype_bytes(y_type))}, {workspace, need}};
    if (!outputs_clear(outs, 2, ins, 6)) return QMM_ERR_UNSUPPORTED;
    LaunchCtx ctx;
    if (!make_ctx(&ctx)) return QMM_ERR_CUDA;
    const ExpertsDown a = {p, static_cast<const uint8_t *>(wd), h, ids, weights, y, workspace, h_stride, y_stride, n, k,
                           h_type == QMM_BF16, y_type == QMM_BF16};
    return from_cuda(launch_experts_down(a, reinterpret_cast<cudaStream_t>(stream), ctx));
}

qmm_status qmm_logits_adjust(const qmm_logits_args *args, qmm_stream_t stream) {
    if (!args) return QMM_ERR_NULL;
    const qmm_logits_args &a = *args;
    if (!a.logits || !a.out) return QMM_ERR_NULL;
    if (a.rows < 1 || a.vocab < 1 || a.logits_stride < a.vocab || a.out_stride < a.vocab ||
        a.history_len < 0 || a.bias_len < 0)
        return QMM_ERR_SHAPE;
    // lists come whole or not at all; an empty list may have no storage
    if ((a.history && !a.hist_start) || (a.hist_start && !a.history && a.history_len > 0) ||
        (a.bias_ids && (!a.bias_values || !a.bias_start)) ||
        (!a.bias_ids && (a.bias_values || (a.bias_start && a.bias_len > 0))))
        return QMM_ERR_NULL;
    if (a.rows > 65535 || a.vocab > kMaxIndex - 65536 || a.history_len > kMaxIndex ||
        a.bias_len > kMaxIndex || a.logits_stride > (int64_t(1) << 40) || a.out_stride > (int64_t(1) << 40))
        return QMM_ERR_UNSUPPORTED;
    for (const void *p : {static_cast<const void *>(a.logits), static_cast<const void *>(a.out),
                          static_cast<const void *>(a.history), static_cast<const void *>(a.hist_start),
                          static_cast<const void *>(a.prompt_len), static_cast<const void *>(a.repetition),
                          static_cast<const void *>(a.frequency), static_cast<const void *>(a.presence),
                          static_cast<const void *>(a.bias_ids), static_cast<const void *>(a.bias_values),
                          static_cast<const void *>(a.bias_start), static_cast<const void *>(a.allowed)})
        if (!aligned(p, 4)) return QMM_ERR_ALIGN;
    const size_t m = static_cast<size_t>(a.rows);
    const bool in_place = a.logits == a.out && a.logits_stride == a.out_stride;
    const Range ins[] = {{in_place ? nullptr : a.logits, rows_bytes(a.rows, a.logits_stride, a.vocab, 4)},
                         {a.history, 4 * static_cast<size_t>(a.history_len)}, {a.hist_start, 4 * (m + 1)},
                         {a.prompt_len, 4 * m}, {a.repetition, 4 * m}, {a.frequency, 4 * m},
                         {a.presence, 4 * m}, {a.bias_ids, 4 * static_cast<size_t>(a.bias_len)},
                         {a.bias_values, 4 * static_cast<size_t>(a.bias_len)}, {a.bias_start, 4 * (m + 1)},
                         {a.allowed, 4 * m * static_cast<size_t>((a.vocab + 31) / 32)}};
    const Range outs[] = {{a.out, rows_bytes(a.rows, a.out_stride, a.vocab, 4)}};
    if (!outputs_clear(outs, 1, ins, 11)) return QMM_ERR_UNSUPPORTED;
    LaunchCtx ctx;
    if (!make_ctx(&ctx)) return QMM_ERR_CUDA;
    const LogitsArgs k = {a.logits, a.out, a.history, a.hist_start, a.prompt_len, a.repetition,
                          a.frequency, a.presence, a.bias_ids, a.bias_values, a.bias_start, a.allowed,
                          a.logits_stride, a.out_stride, a.rows, a.vocab, a.history_len, a.bias_len};
    return from_cuda(launch_logits_adjust(k, reinterpret_cast<cudaStream_t>(stream), ctx));
}

const char *qmm_status_string(qmm_status status) {
    switch (status) {
        case QMM_OK: return "ok";
        case QMM_ERR_NULL: return "null pointer argument";
        case QMM_ERR_SHAPE: return "invalid shape (k % 32 != 0, a size < 1, or m out of range)";
        case QMM_ERR_ALIGN: return "pointer alignment not supported by this call";
        case QMM_ERR_UNSUPPORTED: return "valid arguments not supported by this build";
        case QMM_ERR_CUDA: return "CUDA runtime error";
        case QMM_ERR_TIMEOUT: return "a device-side wait timed out";
        case QMM_ERR_SCRATCH:
            return "problem larger than the entry point's fixed scratch (qmm_gemm_q4_0_prefill: k > 131072)";
        case QMM_ERR_INDEX: return "a page, slot or length on the device lies outside its array";
    }
    return "unknown status";
}

int qmm_version(void) { return 600; }  // 0.6.0: rotation, routing and experts' products added

qmm_status qmm_get_device_error(qmm_stream_t stream) {
    cudaError_t e;
    if (!device_state(&e)) return QMM_ERR_CUDA;
    if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
        return QMM_ERR_CUDA;
    uint32_t word = 0;
    const uint32_t zero = 0;
    if (cudaMemcpyFromSymbol(&word, g_device_error, sizeof word) != cudaSuccess) return QMM_ERR_CUDA;
    if (word != 0 && cudaMemcpyToSymbol(g_device_error, &zero, sizeof zero) != cudaSuccess)
        return QMM_ERR_CUDA;
    return word == 0 ? QMM_OK : static_cast<qmm_status>(word);
}

void qmm_set_wait_timeout_ns(uint64_t ns) {
    g_timeout_ns.store(ns == 0 ? kDefaultTimeoutNs : ns, std::memory_order_relaxed);
}

qmm_status qmm_selftest_wait_timeout(uint64_t timeout_ns, qmm_stream_t stream) {
    LaunchCtx ctx;
    if (!make_ctx(&ctx)) return QMM_ERR_CUDA;
    ctx.timeout_ns = timeout_ns;
    return from_cuda(launch_selftest_wait(reinterpret_cast<cudaStream_t>(stream), ctx));
}

}  // extern "C"
