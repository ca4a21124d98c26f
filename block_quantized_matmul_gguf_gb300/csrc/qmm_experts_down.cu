// qmm_experts_down.cu -- the streaming form's down projections
// (qmm_experts.cuh) and the weighted sums of a token's experts.
#include "qmm_experts.cuh"

namespace qmm {
namespace {

// y[t] = sum_r weights[t][r] z[t topk + r] over the r whose expert is there, in
// their order.  V columns a thread.  z is fp32: rounded to bf16, each projection
// would be off by as much as the result's own rounding.  Bound by the bytes of z,
// which the projections left in L2 where it fits (2047 tokens x 8 to 2048 columns, 134 MB:
// 26 us of the call's 129, 5.5 TB/s with y).
struct SumParams {
    const float *z;
    const int32_t *ids;
    const float *weights;
    void *y;
    int64_t y_stride, tokens, n;
    int experts, topk, parts;  // parts: blocks a token
    bool bf16;  // y
    bool wide;  // y's rows are aligned for V values
};

template <int V>
__device__ __forceinline__ void load_columns(const float *z, float (&f)[V]) {
    if constexpr (V == 1) {
        f[0] = *z;
    } else {
        const float4 v = *reinterpret_cast<const float4 *>(z);
        f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
    }
}

constexpr int kSumAhead = 8;  // rows of z loaded before the first is added

// A block: columns of one token.  A lane reads one pair's expert and weight and the
// warp hands them round.
constexpr int kSumThreads = 128;
template <int V>
__global__ void __launch_bounds__(kSumThreads, 6) sum_kernel(const __grid_constant__ SumParams p) {
    static_assert(V == 1 || V == 4, "a value, or 16 bytes");
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    for (int64_t u = blockIdx.x; u < p.tokens * p.parts; u += gridDim.x) {
        const int64_t t = u / p.parts;
        const int64_t col = (static_cast<int64_t>(u - t * p.parts) * blockDim.x + threadIdx.x) * V;
        const bool mine = col < p.n;  // p.n: a multiple of V
        const float *z = p.z + t * p.topk * p.n + col;
        float sum[V];
#pragma unroll
        for (int v = 0; v < V; ++v) sum[v] = 0.0f;
        for (int r32 = 0; r32 < p.topk; r32 += 32) {
            int id = -1;
            float weight = 0.0f;
            if (r32 + lane < p.topk) {
                id = p.ids[t * p.topk + r32 + lane];
                weight = p.weights[t * p.topk + r32 + lane];
            }
            const uint32_t there = __ballot_sync(0xFFFFFFFFu, id >= 0 && id < p.experts);
            for (int r0 = 0; r0 < 32 && r32 + r0 < p.topk; r0 += kSumAhead) {
                float f[kSumAhead][V];
#pragma unroll
                for (int r = 0; r < kSumAhead; ++r)
                    if (mine && (there >> (r0 + r) & 1)) load_columns<V>(z + (r32 + r0 + r) * p.n, f[r]);
#pragma unroll
                for (int r = 0; r < kSumAhead; ++r) {
                    const float w = __shfl_sync(0xFFFFFFFFu, weight, r0 + r);
                    if (mine && (there >> (r0 + r) & 1))
#pragma unroll
                        for (int v = 0; v < V; ++v) sum[v] = fmaf(w, f[r][v], sum[v]);
                }
            }
        }
        if (!mine) continue;
        if (V == 4 && p.wide) {
            if (p.bf16) {
                uint32_t o[2];
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(sum[2 * v % V], sum[(2 * v + 1) % V]);
                    o[v] = *reinterpret_cast<const uint32_t *>(&b);
                }
                *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.y) + t * p.y_stride + col) = make_uint2(o[0], o[1]);
            } else {
                *reinterpret_cast<float4 *>(static_cast<float *>(p.y) + t * p.y_stride + col) =
                    make_float4(sum[0], sum[1 % V], sum[2 % V], sum[3 % V]);
            }
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) experts::put(p.y, t * p.y_stride + col + v, p.bf16, sum[v]);
        }
    }
}

}  // namespace

// z in front, the rows of h for the tile form behind it.
static size_t z_bytes(int64_t pairs, int64_t n) { return (static_cast<size_t>(pairs) * n * sizeof(float) + 15) & ~size_t(15); }

size_t experts_down_workspace_bytes(int64_t pairs, int64_t n, int64_t k) {
    return z_bytes(pairs, n) + experts_rows_bytes(pairs, k);
}

cudaError_t launch_experts_down(const ExpertsDown &a, cudaStream_t stream, const LaunchCtx &ctx) {
    const bool tiles = experts_tiles_pay(a.plan, a.h, a.h_stride, a.h_bf16 && a.y_bf16, a.n, a.k, false);
    cudaError_t e;
    if (tiles) {
        e = launch_experts_tile_down(a, a.workspace, static_cast<char *>(a.workspace) + z_bytes(a.plan.pairs_total, a.n), stream, ctx);
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
        e = experts::launch_form<false>(p, stream);
    }
    if (e != cudaSuccess) return e;
    const int64_t tokens = a.plan.pairs_total / a.plan.topk;
    const bool whole = a.n % 4 == 0;  // the workspace is aligned
    const int64_t per = whole ? a.n / 4 : a.n;
    const int threads = static_cast<int>(std::min<int64_t>(kSumThreads, (per + 31) / 32 * 32));
    const int parts = static_cast<int>((per + threads - 1) / threads);
    const SumParams s = {static_cast<const float *>(a.workspace), a.ids, a.weights, a.y, a.y_stride, tokens, a.n, a.plan.experts,
                         a.plan.topk, parts, a.y_bf16,
                         reinterpret_cast<uintptr_t>(a.y) % (a.y_bf16 ? 8 : 16) == 0 && a.y_stride % 4 == 0};
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(tokens * parts, int64_t(1) << 30));
    return launch_kernel(whole ? sum_kernel<4> : sum_kernel<1>, dim3(grid), dim3(threads), 0, stream, 1, s);
}

}  // namespace qmm
