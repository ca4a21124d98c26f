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
    int experts, topk, parts;  // parts: blocks a token
    bool bf16;  // y
    bool wide;  // y's rows are aligned to 16 bytes
};

// V columns of a row of z as they are, 16 bytes where V is not 1, and as fp32.
template <typename T, int V>
struct Columns {
    uint4 raw;
    __device__ __forceinline__ void load(const T *z) {
        if constexpr (V == 1)
            raw.x = sizeof(T) == 4 ? __float_as_uint(*reinterpret_cast<const float *>(z)) : *reinterpret_cast<const uint16_t *>(z);
        else
            raw = *reinterpret_cast<const uint4 *>(z);
    }
    __device__ __forceinline__ void add(float w, float (&sum)[V]) const {
        static_assert(V == 1 || V * sizeof(T) == 16, "16 bytes");
        const uint32_t r[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint32_t q = sizeof(T) == 4 ? r[v % 4] : v % 2 ? r[v / 2 % 4] & 0xFFFF0000u : r[v / 2 % 4] << 16;
            sum[v] = fmaf(w, __uint_as_float(q), sum[v]);
        }
    }
};

constexpr int kSumAhead = 8;  // rows of z loaded before the first is added

// A block: columns of one token.  A lane reads one pair's expert and weight and the
// warp hands them round.  Blocks of 128 threads, six an SM or more: the projections of
// 2047 tokens x 8 to 2048 columns 93.2 us in all; 256 threads, without a limit on
// registers (116 of them, two blocks an SM) 97.8, with four blocks an SM 94.8.
constexpr int kSumThreads = 128;
template <typename T, int V>
__global__ void __launch_bounds__(kSumThreads, 6) sum_kernel(const __grid_constant__ SumParams p) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    for (int64_t u = blockIdx.x; u < p.tokens * p.parts; u += gridDim.x) {
        const int64_t t = u / p.parts;
        const int64_t col = (static_cast<int64_t>(u - t * p.parts) * blockDim.x + threadIdx.x) * V;
        const bool mine = col < p.n;  // p.n: a multiple of V
        const T *z = static_cast<const T *>(p.z) + t * p.topk * p.n + col;
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
                Columns<T, V> f[kSumAhead];
#pragma unroll
                for (int r = 0; r < kSumAhead; ++r)
                    if (mine && (there >> (r0 + r) & 1)) f[r].load(z + (r32 + r0 + r) * p.n);
#pragma unroll
                for (int r = 0; r < kSumAhead; ++r) {
                    const float w = __shfl_sync(0xFFFFFFFFu, weight, r0 + r);
                    if (mine && (there >> (r0 + r) & 1)) f[r].add(w, sum);
                }
            }
        }
        if (!mine) continue;
        if (V == 8 && p.bf16 && p.wide) {
            uint32_t o[4];
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(sum[2 * v % V], sum[(2 * v + 1) % V]);
                o[v] = *reinterpret_cast<const uint32_t *>(&b);
            }
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.y) + t * p.y_stride + col) = make_uint4(o[0], o[1], o[2], o[3]);
        } else if (V == 4 && !p.bf16 && p.wide) {
            *reinterpret_cast<float4 *>(static_cast<float *>(p.y) + t * p.y_stride + col) =
                make_float4(sum[0], sum[1 % V], sum[2 % V], sum[3 % V]);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) experts::put(p.y, t * p.y_stride + col + v, p.bf16, sum[v]);
        }
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
    const int values = tiles ? 8 : 4;  // of z in 16 bytes
    const bool whole = a.n % values == 0;  // the workspace is aligned
    const int64_t per = whole ? a.n / values : a.n;
    const int threads = static_cast<int>(std::min<int64_t>(kSumThreads, (per + 31) / 32 * 32));
    const int parts = static_cast<int>((per + threads - 1) / threads);
    const SumParams s = {a.workspace, a.ids, a.weights, a.y, a.y_stride, tokens, a.n, a.plan.experts, a.plan.topk, parts, a.y_bf16,
                         reinterpret_cast<uintptr_t>(a.y) % 16 == 0 && a.y_stride % (a.y_bf16 ? 8 : 4) == 0};
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(tokens * parts, int64_t(1) << 30));
    auto *kernel = tiles ? (whole ? sum_kernel<uint16_t, 8> : sum_kernel<uint16_t, 1>)
                         : (whole ? sum_kernel<float, 4> : sum_kernel<float, 1>);
    return launch_kernel(kernel, dim3(grid), dim3(threads), 0, stream, 1, s);
}

}  // namespace qmm
