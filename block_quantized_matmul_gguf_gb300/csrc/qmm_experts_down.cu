// qmm_experts_down.cu -- the streaming form's down projections
// (qmm_experts.cuh) and the weighted sums of a token's experts.
#include "qmm_experts.cuh"

namespace qmm {
namespace {

// y[t] = sum_r weights[t][r] z[t topk + r] over the r whose expert is there, in
// their order.  V columns a thread.  Bound by the bytes of z, which the
// projections left in L2 where it fits.
struct SumParams {
    const void *z;  // fp32, or bf16 from the tile form
    const int32_t *ids;
    const float *weights;
    void *y;
    int64_t y_stride, tokens, n;
    int experts, topk;
    bool bf16;  // y
};

__device__ __forceinline__ float4 four_at(const float *z) { return *reinterpret_cast<const float4 *>(z); }
__device__ __forceinline__ float4 four_at(const uint16_t *z) {
    const uint2 v = *reinterpret_cast<const uint2 *>(z);
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                       __uint_as_float(v.y & 0xFFFF0000u));
}
__device__ __forceinline__ float one_at(const float *z) { return *z; }
__device__ __forceinline__ float one_at(const uint16_t *z) { return __uint_as_float(static_cast<uint32_t>(*z) << 16); }

template <typename T, int V>
__global__ void __launch_bounds__(256) sum_kernel(SumParams p) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t per = (p.n + V - 1) / V, all = per * p.tokens;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < all; i += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t t = i / per, col = (i - t * per) * V;
        float sum[V];
#pragma unroll
        for (int v = 0; v < V; ++v) sum[v] = 0.0f;
#pragma unroll 4
        for (int r = 0; r < p.topk; ++r) {
            const int64_t pair = t * p.topk + r;
            const int id = p.ids[pair];
            if (id < 0 || id >= p.experts) continue;
            const float w = p.weights[pair];
            const T *z = static_cast<const T *>(p.z) + pair * p.n + col;
            if constexpr (V == 4) {
                const float4 f = four_at(z);
                sum[0] = fmaf(w, f.x, sum[0]);
                sum[1] = fmaf(w, f.y, sum[1]);
                sum[2] = fmaf(w, f.z, sum[2]);
                sum[3] = fmaf(w, f.w, sum[3]);
            } else {
                sum[0] = fmaf(w, one_at(z), sum[0]);
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) experts::put(p.y, t * p.y_stride + col + v, p.bf16, sum[v]);
    }
}

}  // namespace

// z in front, as fp32, or as bf16 with the rows of h behind it.
static size_t tile_z_bytes(int64_t pairs, int64_t n) { return (static_cast<size_t>(pairs) * n * 2 + 15) & ~size_t(15); }

size_t experts_down_workspace_bytes(int64_t pairs, int64_t n, int64_t k) {
    return std::max(static_cast<size_t>(pairs) * n * sizeof(float), tile_z_bytes(pairs, n) + experts_rows_bytes(pairs, k));
}

cudaError_t launch_experts_down(const ExpertsDown &a, cudaStream_t stream, const LaunchCtx &ctx) {
    const bool tiles = experts_tiles_pay(a.plan, a.h, a.h_stride, a.h_bf16 && a.y_bf16, a.n, a.k);
    cudaError_t e;
    if (tiles) {
        e = launch_experts_tile_down(a, a.workspace, static_cast<char *>(a.workspace) + tile_z_bytes(a.plan.pairs_total, a.n), stream, ctx);
    } else {
        experts::StreamParams p = {};
        p.plan = a.plan;
        p.w[0] = p.w[1] = a.wd;
        p.x = a.h;
        p.x_stride = a.h_stride;
        p.x_bf16 = a.h_bf16;
        p.out = a.workspace;
        p.out_stride = a.n;
        p.out_bf16 = false;
        p.n = a.n;
        p.k = a.k;
        p.ctx = ctx;
        e = experts::launch_form<false>(p, !a.y_bf16, stream);
    }
    if (e != cudaSuccess) return e;
    const int64_t tokens = a.plan.pairs_total / a.plan.topk;
    const SumParams s = {a.workspace, a.ids, a.weights, a.y, a.y_stride, tokens, a.n, a.plan.experts,
                         a.plan.topk, a.y_bf16};
    const bool wide = a.n % 4 == 0;  // the workspace is aligned
    const int64_t threads = tokens * (wide ? a.n / 4 : a.n);
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>((threads + 255) / 256, static_cast<int64_t>(device_sm_count()) * 8));
    auto *kernel = tiles ? (wide ? sum_kernel<uint16_t, 4> : sum_kernel<uint16_t, 1>)
                         : (wide ? sum_kernel<float, 4> : sum_kernel<float, 1>);
    return launch_kernel(kernel, dim3(grid), dim3(256), 0, stream, 1, s);
}

}  // namespace qmm
