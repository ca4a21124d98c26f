// qmm_logits.cu -- penalties for repeated tokens, biases and grammar masks on
// the logits of a batch (include/qmm.h, qmm_logits_adjust).
//
// One launch, no workspace: a CTA owns a slice of one row's vocabulary, keeps
// a word per logit of it in shared memory (times generated, and whether the
// prompt or the bias list names it), reads the row's whole history and counts
// the ids that fall into its slice, then passes its logits through once, of
// which only the marked ones take more than a mask.  The counts are integers,
// so the order of the shared atomics does not matter; bias entries are added
// in list order.  Bound by HBM (8 bytes a logit) and the latency of the lists:
// 64 rows of 262143 logits 47 us, of which the stream alone takes 22, the mask
// 5, histories of 8000 ids (read once per slice, from L2) 12 and bias lists of
// 100 entries 4.  Clusters of slices that share a history's reading by remote
// shared atomics took 56 us.
#include "qmm_internal.h"

#include <algorithm>

namespace qmm {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 8;  // list entries a thread has under way
constexpr uint32_t kInPrompt = 0x80000000u, kBiased = 0x40000000u;  // the other bits count what was generated

__device__ __forceinline__ int32_t bounded(int32_t v, int64_t len, bool &bad) {
    const int64_t w = min(max(static_cast<int64_t>(v), int64_t(0)), len);
    bad |= w != v;
    return static_cast<int32_t>(w);
}

// What a CTA keeps of the bias list: the entries of its slice, in list order.
// Beyond kBiasKept of them it sums them by logit instead (add_long_list).
struct BiasEntry {
    int32_t id;
    float value;
};
constexpr int kBiasKept = 512;

// Sum of the kept entries for id, in their order.
__device__ __forceinline__ float bias_of(const BiasEntry *kept, int n, int32_t id) {
    float v = 0.0f;
    for (int i = 0; i < n; ++i)
        if (kept[i].id == id) v += kept[i].value;
    return v;
}

// Adds the entries of the row's list that name an id of the slice (first ..
// first + count - 1, the first at place `shift`) to sums[place], in list order:
// a warp takes the places that are its own number modulo the warps, and of the
// entries of one id among 32 the first one's lane adds all.  262144 entries for
// 262144 logits: 1.3 ms, 46 when every logit read the list for itself.
__device__ __noinline__ void add_long_list(const int32_t *ids, const float *values, int32_t b0, int32_t b1, int32_t first,
                                           uint32_t count, int shift, float *sums) {
    constexpr uint32_t kWarps = kThreads / 32;
    const int lane = threadIdx.x & 31;
    const uint32_t warp = threadIdx.x >> 5;
    for (int64_t b = b0; b < b1; b += 32 * kAhead) {
        int32_t id[kAhead];
        float value[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int64_t i = b + u * 32 + lane;
            id[u] = i < b1 ? ids[i] : -1;
            value[u] = i < b1 ? values[i] : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const uint32_t e = static_cast<uint32_t>(id[u] - first), place = shift + e;
            const bool here = id[u] >= 0 && e < count && place % kWarps == warp;
            if (!__any_sync(0xFFFFFFFFu, here)) continue;
            const unsigned same = __match_any_sync(0xFFFFFFFFu, here ? id[u] : -1);
            const bool leads = here && (same & ((1u << lane) - 1u)) == 0u;
            float sum = leads ? sums[place] + value[u] : 0.0f;
            unsigned rest = leads ? same & (same - 1u) : 0u;  // the others, in their order
            while (__any_sync(0xFFFFFFFFu, rest != 0u)) {
                const int from = rest ? __ffs(rest) - 1 : lane;
                const float v = __shfl_sync(0xFFFFFFFFu, value[u], from);
                if (rest) sum += v;
                rest &= rest - 1u;
            }
            if (leads) sums[place] = sum;
            __syncwarp();
        }
    }
}

// Q float4 per thread: the slice is Q * 1024 logits.  All of them pass through
// at once, with the mask alone; the marked ones are written again when the
// lists have been read, which nothing of the stream then waits for.
template <int Q>
__global__ void __launch_bounds__(kThreads) logits_kernel(const __grid_constant__ LogitsArgs a, LaunchCtx ctx) {
    constexpr int S = Q * 4 * kThreads;
    __shared__ __align__(16) uint32_t seen[S];
    __shared__ uint16_t marked[S];  // places of the marked logits, in any order
    constexpr uint16_t kPlace = 0x7FFF, kHasBias = 0x8000;
    static_assert(S <= kPlace, "a place and a flag");
    __shared__ BiasEntry kept[kBiasKept];
    __shared__ int kept_n, marked_n;
    // all rows' first slices first: low ids are common, and the slices that
    // hold many of a history's take longest
    const int slice = static_cast<int>(blockIdx.x / static_cast<unsigned>(a.rows));
    const int64_t row = blockIdx.x - static_cast<unsigned>(slice) * static_cast<unsigned>(a.rows);
    const float *in = a.logits + row * a.logits_stride;
    float *out = a.out + row * a.out_stride;
    // The slices are cut at 16-byte boundaries of the input: place e of the
    // row is index e + pad.
    const int pad = static_cast<int>((reinterpret_cast<uintptr_t>(in) >> 2) & 3), vocab = static_cast<int>(a.vocab);
    const int base = slice * S - pad;  // the slice's first place
    if (base >= vocab) return;
    const bool wide_out = static_cast<int>((reinterpret_cast<uintptr_t>(out) >> 2) & 3) == pad;
    const bool whole = base >= 0 && base + S <= vocab;
    const int e0 = base + static_cast<int>(threadIdx.x) * 4;  // the thread's first place; then every 4 kThreads
    const float ninf = __uint_as_float(0xFF800000u);

    pdl_wait();
    pdl_launch_dependents();
    // the lists' ends, under way before the stream's loads
    bool bad = false;
    int32_t h0 = 0, h1 = 0, b0 = 0, b1 = 0;
    int64_t made = 0;
    if (a.history) {
        h0 = bounded(a.hist_start[row], a.history_len, bad);
        h1 = bounded(a.hist_start[row + 1], a.history_len, bad);
        made = h0 + static_cast<int64_t>(a.prompt_len ? max(a.prompt_len[row], 0) : 0);
    }
    if (a.bias_ids) {
        b0 = bounded(a.bias_start[row], a.bias_len, bad);
        b1 = bounded(a.bias_start[row + 1], a.bias_len, bad);
    }
    const uint32_t *allowed = a.allowed ? a.allowed + row * ((a.vocab + 31) / 32) : nullptr;
    if (whole) {
        float4 x[Q];
        uint32_t bits[Q];  // of four logits each
#pragma unroll
        for (int i = 0; i < Q; ++i) x[i] = reinterpret_cast<const float4 *>(in + e0)[i * kThreads];
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            bits[i] = 15u;
            if (allowed) {
                const int e = e0 + i * 4 * kThreads;
                const uint32_t w = allowed[e >> 5];
                bits[i] = __funnelshift_r(w, pad ? allowed[(e + 3) >> 5] : w, e & 31);
            }
        }
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            float4 y = x[i];
            if (!(bits[i] & 1u)) y.x = ninf;
            if (!(bits[i] & 2u)) y.y = ninf;
            if (!(bits[i] & 4u)) y.z = ninf;
            if (!(bits[i] & 8u)) y.w = ninf;
            if (wide_out) {
                __stcs(reinterpret_cast<float4 *>(out + e0) + i * kThreads, y);
            } else {
                float *to = out + e0 + i * 4 * kThreads;
                to[0] = y.x, to[1] = y.y, to[2] = y.z, to[3] = y.w;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < Q; ++i) {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int e = e0 + i * 4 * kThreads + t;
                if (e >= 0 && e < vocab)
                    out[e] = !allowed || ((allowed[e >> 5] >> (e & 31)) & 1u) ? in[e] : ninf;
            }
        }
    }
    if (!a.history && !a.bias_ids) return;

    // ids of the slice: first .. first + count - 1, the first at place `shift`
    const int first = max(base, 0), shift = first - base;
    const uint32_t count = static_cast<uint32_t>(min(base + S, vocab) - first);
#pragma unroll
    for (int i = 0; i < Q; ++i)
        *reinterpret_cast<uint4 *>(seen + (i * kThreads + threadIdx.x) * 4) = make_uint4(0u, 0u, 0u, 0u);
    if (threadIdx.x == 0) {
        marked_n = 0;
        if (bad) record_error(ctx, kDevErrIndex);
    }
    int32_t id[kAhead];
    auto load_ids = [&](const int32_t *list, int64_t from, int32_t end, int step, int lane) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int64_t i = from + u * step + lane;
            id[u] = i < end ? list[i] : -1;
        }
    };
    // the last warp reads the bias list, the others the history
    const int readers = a.bias_ids ? kThreads - 32 : kThreads, lane = threadIdx.x & 31;
    const bool bias_warp = static_cast<int>(threadIdx.x) >= readers;
    if (bias_warp)
        load_ids(a.bias_ids, b0, b1, 32, lane);
    else
        load_ids(a.history, h0, h1, readers, threadIdx.x);
    auto mark = [&](uint32_t e, uint32_t old) {  // the first mark of a logit lists it
        if (!old) marked[atomicAdd(&marked_n, 1)] = static_cast<uint16_t>(e);
    };
    __syncthreads();
    if (bias_warp) {
        int n = 0;
        for (int64_t b = b0; b < b1; b += 32 * kAhead) {
            if (b > b0) load_ids(a.bias_ids, b, b1, 32, lane);
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const uint32_t e = static_cast<uint32_t>(id[u] - first);
                const bool here = id[u] >= 0 && e < count;
                const unsigned all = __ballot_sync(0xFFFFFFFFu, here);
                const int at = n + __popc(all & ((1u << lane) - 1u));
                if (here) {
                    mark(shift + e, atomicOr(seen + shift + e, kBiased));
                    if (at < kBiasKept) kept[at] = BiasEntry{id[u], a.bias_values[b + u * 32 + lane]};
                }
                n += __popc(all);
            }
        }
        if (lane == 0) kept_n = n;
    } else {
        for (int64_t h = h0; h < h1; h += static_cast<int64_t>(readers) * kAhead) {
            if (h > h0) load_ids(a.history, h, h1, readers, threadIdx.x);
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const uint32_t e = static_cast<uint32_t>(id[u] - first);  // ids below 0 lie far off
                if (id[u] >= 0 && e < count) {
                    const bool late = h + u * readers + threadIdx.x >= made;
                    mark(shift + e, late ? atomicAdd(seen + shift + e, 1u) : atomicOr(seen + shift + e, kInPrompt));
                }
            }
        }
    }
    const float rep = a.repetition ? a.repetition[row] : 1.0f;
    const float freq = a.frequency ? a.frequency[row] : 0.0f;
    const float pres = a.presence ? a.presence[row] : 0.0f;
    __syncthreads();
    const bool long_list = a.bias_ids && kept_n > kBiasKept;
    for (int i = threadIdx.x; i < marked_n; i += kThreads) {
        const int at = marked[i] & kPlace, e = base + at;
        const uint32_t mark = seen[at], n = mark & ~(kInPrompt | kBiased);
        if (long_list && (mark & kBiased)) marked[i] |= kHasBias;
        if (allowed && !((allowed[e >> 5] >> (e & 31)) & 1u)) continue;  // masked for good
        float y = in[e];  // in place: its own value still, as the mask left it alone
        if (n || (mark & kInPrompt)) {
            if (a.repetition) y = y > 0.0f ? __fdiv_rn(y, rep) : y * rep;
            y -= __fmul_rn(static_cast<float>(n), freq) + (n ? pres : 0.0f);
        }
        if ((mark & kBiased) && !long_list) y += bias_of(kept, kept_n, e);
        out[e] = y;
    }
    if (!long_list) return;
    // the marks have been read: their places take the sums
    __syncthreads();
    float *sums = reinterpret_cast<float *>(seen);
    for (int i = threadIdx.x; i < marked_n; i += kThreads) sums[marked[i] & kPlace] = 0.0f;
    __syncthreads();
    add_long_list(a.bias_ids, a.bias_values, b0, b1, first, count, shift, sums);
    __syncthreads();
    for (int i = threadIdx.x; i < marked_n; i += kThreads) {
        const int at = marked[i] & kPlace, e = base + at;
        if (!(marked[i] & kHasBias) || (allowed && !((allowed[e >> 5] >> (e & 31)) & 1u))) continue;
        out[e] += sums[at];
    }
}

template <int Q>
cudaError_t launch_slices(const LogitsArgs &a, cudaStream_t stream, const LaunchCtx &ctx) {
    constexpr int S = Q * 4 * kThreads;
    const unsigned slices = static_cast<unsigned>((a.vocab + 3 + S - 1) / S);  // + 3: the padding
    return launch_kernel(logits_kernel<Q>, dim3(slices * static_cast<unsigned>(a.rows)), dim3(kThreads), 0, stream, 1, a,
                         ctx);
}

}  // namespace

cudaError_t launch_logits_adjust(const LogitsArgs &a, cudaStream_t stream, const LaunchCtx &ctx) {
    // Long slices read each history fewer times; short ones spread a few rows
    // over the whole GPU.  GPU time with slices of 2048 / 4096 logits, vocabulary
    // 262144: 1 row 3.2 / 3.8 us, 4 rows 4.9 / 4.4, 16 rows 9.4 / 8.3; 64 rows
    // with histories of 8000, 58 / 47, and 59 with slices of 8192.
    if (a.rows * ((a.vocab + 4095) / 4096) >= device_sm_count()) return launch_slices<4>(a, stream, ctx);
    return launch_slices<2>(a, stream, ctx);
}

}  // namespace qmm
