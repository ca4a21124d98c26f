// qmm_logits.cu -- penalties for repeated tokens, biases and grammar masks on
// the logits of a batch (include/qmm.h, qmm_logits_adjust).
//
// One launch, no workspace: a CTA owns a slice of one row's vocabulary, keeps
// that slice's token counts (and bias sums) in shared memory, reads the row's
// whole history and counts the ids that fall into its slice, then passes its
// logits through once.  The counts are integers, so the order of the shared
// atomics does not matter; bias entries are added by one warp in list order.
// Bound by HBM (8 bytes a logit); the histories are read once per slice, from
// L2, so rows with long histories get larger slices.
#include "qmm_internal.h"

#include <algorithm>

namespace qmm {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 8;  // history entries a thread has under way
constexpr uint32_t kInPrompt = 0x80000000u;  // the other bits count what was generated

__device__ __forceinline__ int32_t bounded(int32_t v, int64_t len, bool &bad) {
    const int64_t w = min(max(static_cast<int64_t>(v), int64_t(0)), len);
    bad |= w != v;
    return static_cast<int32_t>(w);
}

// Q float4 per thread: the slice is Q * 1024 logits.
template <int Q>
__global__ void __launch_bounds__(kThreads) logits_kernel(LogitsArgs a, LaunchCtx ctx) {
    constexpr int S = Q * 4 * kThreads;
    extern __shared__ uint32_t seen[];                       // [S] if there is a history
    float *bias = reinterpret_cast<float *>(seen + (a.history ? S : 0));  // [S] if there is a bias
    const int64_t row = blockIdx.y;
    const float *in = a.logits + row * a.logits_stride;
    float *out = a.out + row * a.out_stride;
    // The slices are cut at 16-byte boundaries of the input: place e of the
    // row is index e + pad.
    const int pad = static_cast<int>((reinterpret_cast<uintptr_t>(in) >> 2) & 3);
    const int64_t base = static_cast<int64_t>(blockIdx.x) * S - pad;  // the slice's first place
    if (base >= a.vocab) return;
    const bool wide_out = ((reinterpret_cast<uintptr_t>(out) >> 2) & 3) == pad;

    pdl_wait();
    pdl_launch_dependents();
    float4 x[Q];
#pragma unroll
    for (int i = 0; i < Q; ++i) {
        const int64_t e = base + (i * kThreads + threadIdx.x) * 4;
        if (e >= 0 && e + 4 <= a.vocab) {
            x[i] = *reinterpret_cast<const float4 *>(in + e);
        } else {
            x[i].x = e >= 0 && e < a.vocab ? in[e] : 0.0f;
            x[i].y = e + 1 >= 0 && e + 1 < a.vocab ? in[e + 1] : 0.0f;
            x[i].z = e + 2 >= 0 && e + 2 < a.vocab ? in[e + 2] : 0.0f;
            x[i].w = e + 3 >= 0 && e + 3 < a.vocab ? in[e + 3] : 0.0f;
        }
    }
    const int used = (a.history ? S : 0) + (a.bias_ids ? S : 0);
    for (int i = threadIdx.x * 4; i < used; i += kThreads * 4)
        *reinterpret_cast<uint4 *>(seen + i) = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
    bool bad = false;
    if (a.history) {
        const int32_t h0 = bounded(a.hist_start[row], a.history_len, bad);
        const int32_t h1 = bounded(a.hist_start[row + 1], a.history_len, bad);
        const int64_t made = h0 + static_cast<int64_t>(a.prompt_len ? max(a.prompt_len[row], 0) : 0);
        const int first = static_cast<int>(max(base, int64_t(0))), count = static_cast<int>(min(base + S, a.vocab)) - first;
        const int shift = static_cast<int>(first - base);
        for (int64_t h = h0; h < h1; h += kThreads * kAhead) {
            int32_t id[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int64_t i = h + u * kThreads + threadIdx.x;
                id[u] = i < h1 ? a.history[i] : -1;
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const uint32_t e = static_cast<uint32_t>(id[u]) - static_cast<uint32_t>(first);
                if (e < static_cast<uint32_t>(count)) {  // also false for ids below 0
                    if (h + u * kThreads + threadIdx.x < made)
                        atomicOr(seen + shift + e, kInPrompt);
                    else
                        atomicAdd(seen + shift + e, 1u);
                }
            }
        }
    }
    if (a.bias_ids && threadIdx.x < 32) {
        const int32_t b0 = bounded(a.bias_start[row], a.bias_len, bad);
        const int32_t b1 = bounded(a.bias_start[row + 1], a.bias_len, bad);
        for (int64_t b = b0; b < b1; b += 32) {
            const int64_t i = b + threadIdx.x;
            int64_t e = -1;
            float v = 0.0f;
            if (i < b1) {
                const int64_t id = a.bias_ids[i];
                if (id >= 0 && id < a.vocab && id >= base && id < base + S) e = id - base;
                v = a.bias_values[i];
            }
            // in list order: the entries of one id one after another
            unsigned todo = __ballot_sync(0xFFFFFFFFu, e >= 0);
            while (todo) {
                const int from = __ffs(todo) - 1;
                if (static_cast<int>(threadIdx.x) == from) bias[e] += v;
                __syncwarp();
                todo &= todo - 1;
            }
        }
    }
    if (bad && threadIdx.x == 0) record_error(ctx, kDevErrIndex);
    __syncthreads();
    const float rep = a.repetition ? a.repetition[row] : 1.0f;
    const float freq = a.frequency ? a.frequency[row] : 0.0f;
    const float pres = a.presence ? a.presence[row] : 0.0f;
    const uint32_t *allowed = a.allowed ? a.allowed + row * ((a.vocab + 31) / 32) : nullptr;
#pragma unroll
    for (int i = 0; i < Q; ++i) {
        const int at = (i * kThreads + threadIdx.x) * 4;
        const int64_t e = base + at;
        float y[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        if (a.history) {
            const uint4 s4 = *reinterpret_cast<const uint4 *>(seen + at);
            const uint32_t s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                if (s[t]) {  // few logits were seen
                    if (a.repetition) y[t] = y[t] > 0.0f ? __fdiv_rn(y[t], rep) : y[t] * rep;
                    const uint32_t c = s[t] & ~kInPrompt;
                    y[t] -= __fmul_rn(static_cast<float>(c), freq) + (c ? pres : 0.0f);
                }
            }
        }
        if (a.bias_ids) {
            const float4 b = *reinterpret_cast<const float4 *>(bias + at);
            y[0] += b.x;
            y[1] += b.y;
            y[2] += b.z;
            y[3] += b.w;
        }
        if (allowed) {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int64_t f = e + t;
                if (f >= 0 && f < a.vocab && !((allowed[f >> 5] >> (f & 31)) & 1u))
                    y[t] = __uint_as_float(0xFF800000u);
            }
        }
        if (wide_out && e >= 0 && e + 4 <= a.vocab) {
            *reinterpret_cast<float4 *>(out + e) = make_float4(y[0], y[1], y[2], y[3]);
        } else {
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (e + t >= 0 && e + t < a.vocab) out[e + t] = y[t];
        }
    }
}

template <int Q>
cudaError_t launch_slices(const LogitsArgs &a, cudaStream_t stream, const LaunchCtx &ctx) {
    constexpr int S = Q * 4 * kThreads;
    static int limits[kMaxDevices];
    const size_t smem = sizeof(uint32_t) * S * ((a.history ? 1 : 0) + (a.bias_ids ? 1 : 0));
    if (smem > 48 * 1024) {
        const cudaError_t e = ensure_smem(logits_kernel<Q>, smem, false, limits);
        if (e != cudaSuccess) return e;
    }
    const unsigned slices = static_cast<unsigned>((a.vocab + 3 + S - 1) / S);  // + 3: the padding
    return launch_kernel(logits_kernel<Q>, dim3(slices, static_cast<unsigned>(a.rows)), dim3(kThreads),
                         smem, stream, 1, a, ctx);
}

}  // namespace

cudaError_t launch_logits_adjust(const LogitsArgs &a, cudaStream_t stream, const LaunchCtx &ctx) {
    // Long slices read each history fewer times; short ones spread a few
    // rows over the whole GPU.
    const int64_t wide = a.rows * ((a.vocab + 8191) / 8192);
    if (wide >= 2 * device_sm_count()) return launch_slices<8>(a, stream, ctx);
    return launch_slices<2>(a, stream, ctx);
}

}  // namespace qmm
