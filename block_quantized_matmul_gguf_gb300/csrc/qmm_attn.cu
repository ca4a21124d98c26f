// qmm_attn.cu -- attention over the paged Q4_0 cache (include/qmm.h,
// qmm_attn_q4_0).
//
// One CTA per query row and head: each of its four warps takes every fourth
// key, keeps the running maximum and sum of the softmax and its share of the
// output, and the warps' shares are joined at the end.  A lane holds the
// values of head_dim / 64 code bytes of a key, the same bytes for every key.
#include "qmm_internal.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace qmm {
namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ float load_one(const void *p, int64_t i, bool bf16) {
    if (bf16)
        return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(p)[i]) << 16);
    return static_cast<const float *>(p)[i];
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) attn_row_kernel(AttnArgs a, KvCache c, LaunchCtx ctx) {
    constexpr int B = D / 64;  // code bytes per lane
    pdl_wait();
    pdl_launch_dependents();
    const int64_t row = blockIdx.x;
    const int head = blockIdx.y;
    if (row == 0 && head == 0 && threadIdx.x == 0 && a.q_start[a.batch] > a.total_q)
        record_error(ctx, kDevErrIndex);
    if (row >= a.q_start[a.batch] || row < a.q_start[0]) return;
    int lo = 0, hi = a.batch;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.q_start[mid] <= row)
            lo = mid;
        else
            hi = mid;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    bool bad = false;
    int64_t len = max(a.kv_len[lo], 0);
    const int64_t pos = len - (a.q_start[lo + 1] - row);
    bad |= a.q_start[lo + 1] - a.q_start[lo] > a.max_q;
    if (len > (a.table_width << c.page_shift)) {
        len = a.table_width << c.page_shift;
        bad = true;
    }
    const int64_t end = a.causal ? min(len, pos + 1) : len;
    const int64_t begin = a.window ? max(int64_t(0), pos - a.window + 1) : 0;
    float q[2 * B], o[2 * B];
#pragma unroll
    for (int i = 0; i < B; ++i) {
        const int byte = lane + 32 * i;
        const int64_t at = row * a.q_stride + head * D + (byte >> 4) * 32 + (byte & 15);
        q[2 * i] = load_one(a.q, at, a.q_bf16);
        q[2 * i + 1] = load_one(a.q, at + 16, a.q_bf16);
        o[2 * i] = o[2 * i + 1] = 0.0f;
    }
    const int kv_head = head / (a.heads / c.kv_heads);
    const uint8_t *kc = static_cast<const uint8_t *>(c.k_codes), *vc = static_cast<const uint8_t *>(c.v_codes);
    const __half *ks = static_cast<const __half *>(c.k_scales), *vs = static_cast<const __half *>(c.v_scales);
    const float ninf = __uint_as_float(0xFF800000u);
    float m = ninf, l = 0.0f;
    for (int64_t j = begin + warp; j < end; j += kWarps) {
        const int32_t page = a.table[lo * a.table_width + (j >> c.page_shift)];
        if (page < 0 || page >= c.num_pages) {
            bad = true;
            continue;
        }
        const int64_t r = ((static_cast<int64_t>(page) * c.kv_heads + kv_head) << c.page_shift) +
                          (j & ((int64_t(1) << c.page_shift) - 1));
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < B; ++i) {
            const int byte = lane + 32 * i;
            const uint32_t w = kc[r * (D / 2) + byte];
            const float d = __half2float(ks[r * (D / 32) + (byte >> 4)]);
            s = fmaf(q[2 * i], (static_cast<float>(w & 15u) - 8.0f) * d, s);
            s = fmaf(q[2 * i + 1], (static_cast<float>(w >> 4) - 8.0f) * d, s);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
        s *= a.scale;
        const float mn = fmaxf(m, s);
        const float ref = mn == ninf ? 0.0f : mn;
        const float f = expf(m - ref), w = expf(s - ref);
        m = mn;
        l = fmaf(l, f, w);
#pragma unroll
        for (int i = 0; i < B; ++i) {
            const int byte = lane + 32 * i;
            const uint32_t b = vc[r * (D / 2) + byte];
            const float d = __half2float(vs[r * (D / 32) + (byte >> 4)]);
            o[2 * i] = fmaf(o[2 * i], f, w * ((static_cast<float>(b & 15u) - 8.0f) * d));
            o[2 * i + 1] = fmaf(o[2 * i + 1], f, w * ((static_cast<float>(b >> 4) - 8.0f) * d));
        }
    }
    __shared__ float share[kWarps][D];
    __shared__ float stat[kWarps][2];
#pragma unroll
    for (int i = 0; i < B; ++i) {
        const int byte = lane + 32 * i;
        share[warp][(byte >> 4) * 32 + (byte & 15)] = o[2 * i];
        share[warp][(byte >> 4) * 32 + (byte & 15) + 16] = o[2 * i + 1];
    }
    if (lane == 0) {
        stat[warp][0] = m;
        stat[warp][1] = l;
        if (bad) record_error(ctx, kDevErrIndex);
    }
    __syncthreads();
    float top = ninf, sum = 0.0f, f[kWarps];
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, stat[w][0]);
    for (int w = 0; w < kWarps; ++w) {
        f[w] = top == ninf ? 0.0f : expf(stat[w][0] - top);
        sum = fmaf(f[w], stat[w][1], sum);
    }
    for (int d = threadIdx.x; d < D; d += kWarps * 32) {
        float y = 0.0f;
        for (int w = 0; w < kWarps; ++w) y = fmaf(f[w], share[w][d], y);
        if (top != ninf) y /= sum;
        const int64_t at = row * a.out_stride + head * D + d;
        if (a.out_bf16)
            static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(y);
        else
            static_cast<float *>(a.out)[at] = y;
    }
    if (a.lse && threadIdx.x == 0) a.lse[row * a.heads + head] = top == ninf ? ninf : top + logf(sum);
}

}  // namespace

size_t attn_workspace_bytes(const KvCache &, int) { return 0; }

cudaError_t launch_attn(const KvCache &c, const AttnArgs &a, cudaStream_t stream, const LaunchCtx &ctx) {
    auto *kernel = c.head_dim == 64 ? attn_row_kernel<64> : c.head_dim == 128 ? attn_row_kernel<128> : attn_row_kernel<256>;
    return launch_kernel(kernel, dim3(static_cast<unsigned>(a.total_q), a.heads), dim3(kWarps * 32), 0, stream, 1, a, c, ctx);
}

}  // namespace qmm
