// qmm_kv.cu -- the paged Q4_0 cache of keys and values: page tables and slot
// maps from request lengths (plan), quantization into the cache (append) and
// reading it back (read).  Layout and formulas: include/qmm.h.
#include "qmm_internal.h"

#include <cuda_fp16.h>

#include <algorithm>

namespace qmm {
namespace {

constexpr int kThreads = 256;

// ---- plan ------------------------------------------------------------------
// q_start and the first free page of each request are exclusive prefix sums
// over the batch; a token then finds its request by bisection.  Bound by
// latency (12 bytes a token out): one launch, in which every CTA forms both
// prefix sums of the whole batch for itself in shared memory (at most 16384
// requests, 128 KB), so that no CTA waits for another.

// Exclusive prefix over the CTA's threads of a pair of sums; returns the totals.
__device__ __forceinline__ void block_exclusive(int64_t &a, int64_t &b, int64_t &total_a,
                                                int64_t &total_b) {
    __shared__ int64_t wa[kThreads / 32], wb[kThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t ia = a, ib = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t ua = __shfl_up_sync(0xFFFFFFFFu, ia, o);
        const int64_t ub = __shfl_up_sync(0xFFFFFFFFu, ib, o);
        if (lane >= o) {
            ia += ua;
            ib += ub;
        }
    }
    if (lane == 31) {
        wa[warp] = ia;
        wb[warp] = ib;
    }
    __syncthreads();
    int64_t pa = 0, pb = 0;
    total_a = total_b = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) {
            pa += wa[w];
            pb += wb[w];
        }
        total_a += wa[w];
        total_b += wb[w];
    }
    a = pa + ia - a;
    b = pb + ib - b;
}

struct PlanParams {
    const int32_t *cached, *added, *free_pages;
    int32_t *table, *q_start, *kv_len, *positions, *taken;
    int64_t *slots;
    int64_t num_free, table_width, capacity;
    int batch, page_shift;
    LaunchCtx ctx;
};

__global__ void __launch_bounds__(kThreads) plan_kernel(PlanParams p) {
    extern __shared__ int32_t plan_smem[];
    int32_t *start = plan_smem;                // [batch + 1]: first token, at most capacity
    int32_t *first = plan_smem + p.batch + 1;  // [batch]: first entry of free_pages
    pdl_wait();
    pdl_launch_dependents();
    const int64_t round = (int64_t(1) << p.page_shift) - 1;
    const int per = (p.batch + kThreads - 1) / kThreads;
    const int b0 = min(p.batch, static_cast<int>(threadIdx.x) * per), b1 = min(p.batch, b0 + per);
    int64_t tokens = 0, pages = 0;
    bool bad = false;
    for (int b = b0; b < b1; ++b) {
        const int32_t c = p.cached[b], a = p.added[b];
        bad |= c < 0 || a < 0;
        const int64_t had = max(c, 0), now = had + max(a, 0);
        tokens += now - had;
        pages += ((now + round) >> p.page_shift) - ((had + round) >> p.page_shift);
    }
    int64_t all_tokens, all_pages;
    block_exclusive(tokens, pages, all_tokens, all_pages);
    for (int b = b0; b < b1; ++b) {
        const int64_t had = max(p.cached[b], 0), now = had + max(p.added[b], 0);
        start[b] = static_cast<int32_t>(min(tokens, p.capacity));
        first[b] = static_cast<int32_t>(min(pages, p.num_free));
        const int64_t page0 = (had + round) >> p.page_shift, page1 = (now + round) >> p.page_shift;
        if (blockIdx.x == 0) {
            p.q_start[b] = start[b];
            bad |= now > INT32_MAX || page1 > p.table_width;
            p.kv_len[b] = static_cast<int32_t>(min(now, static_cast<int64_t>(INT32_MAX)));
        }
        tokens += now - had;
        pages += page1 - page0;
    }
    if (threadIdx.x == 0) {
        start[p.batch] = static_cast<int32_t>(min(all_tokens, p.capacity));
        if (blockIdx.x == 0) {
            p.q_start[p.batch] = start[p.batch];
            p.taken[0] = static_cast<int32_t>(min(all_pages, static_cast<int64_t>(INT32_MAX)));
            bad |= all_tokens > p.capacity || all_pages > p.num_free;
        }
    }
    if (bad && blockIdx.x == 0) record_error(p.ctx, kDevErrIndex);
    __syncthreads();

    const int lane = threadIdx.x & 31;
    const int warps = gridDim.x * (kThreads / 32);
    for (int b = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); b < p.batch; b += warps) {
        const int64_t had = max(p.cached[b], 0), now = had + max(p.added[b], 0);
        const int64_t page0 = (had + round) >> p.page_shift;
        const int64_t page1 = min((now + round) >> p.page_shift, p.table_width);
        for (int64_t i = page0 + lane; i < page1; i += 32) {
            const int64_t at = first[b] + (i - page0);
            p.table[b * p.table_width + i] = at < p.num_free ? p.free_pages[at] : -1;
        }
    }

    const int real = start[p.batch];
    const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; t < p.capacity;
         t += step) {
        int64_t slot = -1;
        int32_t pos = -1;
        if (t < real) {
            int lo = 0, hi = p.batch;  // start[lo] <= t < start[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (start[mid] <= t)
                    lo = mid;
                else
                    hi = mid;
            }
            const int64_t had = max(p.cached[lo], 0);
            const int64_t at = had + (t - start[lo]);
            const int64_t index = at >> p.page_shift, page0 = (had + round) >> p.page_shift;
            int32_t page = -1;
            if (index < p.table_width) {
                const int64_t f = first[lo] + (index - page0);
                if (index < page0)
                    page = p.table[lo * p.table_width + index];  // held before: not written here
                else if (f < p.num_free)
                    page = p.free_pages[f];
            }
            if (page >= 0) slot = (static_cast<int64_t>(page) << p.page_shift) + (at & round);
            pos = static_cast<int32_t>(min(at, static_cast<int64_t>(INT32_MAX)));
        }
        p.slots[t] = slot;
        p.positions[t] = pos;
    }
}

// ---- append ------------------------------------------------------------------
// Eight lanes share a block of 32 values, four each (one 16- or 8-byte load);
// the extremes meet by shuffles, lanes 0-3 take the codes of lanes 4-7 as
// their high nibbles and write the block's 16 bytes.  Bound by the bytes of
// the inputs; a decode step's few blocks are bound by latency.

struct KvView {
    uint8_t *codes[2];
    __half *scales[2];
    int64_t slots;  // of the whole cache
    int page_shift, kv_heads;
};

// Row (page, head, place) of a slot, in rows of head_dim values.
__device__ __forceinline__ int64_t cache_row(const KvView &c, int64_t slot, int head) {
    const int64_t place = slot & ((int64_t(1) << c.page_shift) - 1);
    return ((((slot >> c.page_shift) * c.kv_heads) + head) << c.page_shift) + place;
}

__device__ __forceinline__ float4 load_quad(const float *p, bool wide) {
    if (wide) return *reinterpret_cast<const float4 *>(p);
    return make_float4(p[0], p[1], p[2], p[3]);
}
__device__ __forceinline__ float4 load_quad(const uint16_t *p, bool wide) {
    uint32_t lo, hi;
    if (wide) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        lo = v.x;
        hi = v.y;
    } else {
        lo = p[0] | (static_cast<uint32_t>(p[1]) << 16);
        hi = p[2] | (static_cast<uint32_t>(p[3]) << 16);
    }
    return make_float4(__uint_as_float(lo << 16), __uint_as_float(lo & 0xFFFF0000u),
                       __uint_as_float(hi << 16), __uint_as_float(hi & 0xFFFF0000u));
}

// round(x / d) + 8 within 0..15, IEEE division and rounding to even
__device__ __forceinline__ uint32_t code_of(float x, float d) {
    const float r = rintf(__fdiv_rn(x, d)) + 8.0f;
    return static_cast<uint32_t>(fminf(fmaxf(r, 0.0f), 15.0f));
}

template <typename T>
__global__ void __launch_bounds__(kThreads) append_kernel(KvView c, const T *__restrict__ k,
                                                          int64_t k_stride,
                                                          const T *__restrict__ v,
                                                          int64_t v_stride,
                                                          const int64_t *__restrict__ slots,
                                                          int64_t n, int dim, int wide,
                                                          LaunchCtx ctx) {
    pdl_wait();
    pdl_launch_dependents();
    const int quads = c.kv_heads * dim / 4;  // of a token's keys (or values): a multiple of 16
    const int64_t total = n * 2 * quads;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
    // eight consecutive threads hold one block and leave the loop together
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total; i += step) {
        const int64_t token = i / (2 * quads);
        int at = static_cast<int>(i - token * (2 * quads));
        const int half = at >= quads;
        at -= half * quads;
        const int64_t slot = slots[token];
        const bool live = slot >= 0 && slot < c.slots;
        if (!live && slot != -1) record_error(ctx, kDevErrIndex);
        const unsigned group = 0xFFu << (threadIdx.x & 24);
        if (!live) continue;  // the whole block together
        const T *src = half ? v + token * v_stride : k + token * k_stride;
        const float4 x = load_quad(src + at * 4, wide);
        float top = fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w));
        float low = fminf(fminf(x.x, x.y), fminf(x.z, x.w));
        // 0 * x is NaN for the values that a block cannot hold
        float odd = 0.0f * x.x + 0.0f * x.y + (0.0f * x.z + 0.0f * x.w);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) {
            top = fmaxf(top, __shfl_xor_sync(group, top, o));
            low = fminf(low, __shfl_xor_sync(group, low, o));
            odd += __shfl_xor_sync(group, odd, o);
        }
        const float e = top >= -low ? top : low;
        const __half dh = __float2half_rn(fminf(fmaxf(e * -0.125f, -65504.0f), 65504.0f));
        const float d = __half2float(dh);
        uint32_t q = 0x08080808u;
        const bool finite = odd == 0.0f;
        if (finite && d != 0.0f)
            q = code_of(x.x, d) | (code_of(x.y, d) << 8) | (code_of(x.z, d) << 16) |
                (code_of(x.w, d) << 24);
        const uint32_t high = __shfl_down_sync(group, q, 4, 8);
        const int lane8 = threadIdx.x & 7;
        const int head = at * 4 / dim, block = (at * 4 - head * dim) / kQK;
        const int64_t row = cache_row(c, slot, head);
        if (lane8 < 4)
            *reinterpret_cast<uint32_t *>(c.codes[half] + row * (dim / 2) + block * 16 + lane8 * 4) =
                q | (high << 4);
        if (lane8 == 0)
            c.scales[half][row * (dim / kQK) + block] =
                finite ? dh : __ushort_as_half(static_cast<unsigned short>(0x7FFF));
    }
}

// ---- read ----------------------------------------------------------------------
// Eight lanes share a block, four consecutive values each (as dequant).
// kWide: both outputs are 16-byte aligned.
template <bool kWide>
__global__ void __launch_bounds__(kThreads) read_kernel(KvView c, const int64_t *__restrict__ slots,
                                                        int64_t n, int dim, float *__restrict__ k_out,
                                                        float *__restrict__ v_out, LaunchCtx ctx) {
    pdl_wait();
    pdl_launch_dependents();
    const int quads = c.kv_heads * dim / 4;
    const int64_t total = n * quads;
    const int half = blockIdx.y;
    float *out = half ? v_out : k_out;
    if (!out) return;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total; i += step) {
        const int64_t token = i / quads;
        const int at = static_cast<int>(i - token * quads) * 4;
        const int64_t slot = slots[token];
        float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (slot >= 0 && slot < c.slots) {
            const int head = at / dim, in = at - head * dim;
            const int64_t row = cache_row(c, slot, head);
            const int j = in & 15;
            const uint32_t w = *reinterpret_cast<const uint32_t *>(c.codes[half] + row * (dim / 2) +
                                                                   (in / kQK) * 16 + j) >>
                               ((in & 16) ? 4 : 0);
            const float d = __half2float(c.scales[half][row * (dim / kQK) + in / kQK]);
            y.x = (static_cast<float>(w & 15u) - 8.0f) * d;
            y.y = (static_cast<float>((w >> 8) & 15u) - 8.0f) * d;
            y.z = (static_cast<float>((w >> 16) & 15u) - 8.0f) * d;
            y.w = (static_cast<float>((w >> 24) & 15u) - 8.0f) * d;
        } else if (slot != -1) {
            record_error(ctx, kDevErrIndex);
        }
        float *dst = out + i * 4;
        if constexpr (kWide) {
            *reinterpret_cast<float4 *>(dst) = y;
        } else {
            dst[0] = y.x;
            dst[1] = y.y;
            dst[2] = y.z;
            dst[3] = y.w;
        }
    }
}

KvView view(const KvCache &c) {
    KvView v;
    v.codes[0] = static_cast<uint8_t *>(c.k_codes);
    v.codes[1] = static_cast<uint8_t *>(c.v_codes);
    v.scales[0] = static_cast<__half *>(c.k_scales);
    v.scales[1] = static_cast<__half *>(c.v_scales);
    v.slots = c.num_pages << c.page_shift;
    v.page_shift = c.page_shift;
    v.kv_heads = c.kv_heads;
    return v;
}

unsigned grid_for(int64_t threads, int per_sm) {
    const int64_t cap = static_cast<int64_t>(device_sm_count()) * per_sm;
    return static_cast<unsigned>(std::min((threads + kThreads - 1) / kThreads, cap));
}

}  // namespace

cudaError_t launch_kv_plan(const KvPlan &a, cudaStream_t stream, const LaunchCtx &ctx) {
    static int limits[kMaxDevices];
    const size_t smem = sizeof(int32_t) * (2 * static_cast<size_t>(a.batch) + 1);
    if (smem > 48 * 1024) {
        const cudaError_t e = ensure_smem(plan_kernel, smem, false, limits);
        if (e != cudaSuccess) return e;
    }
    // a CTA reads the whole batch's lengths, so it takes 2048 tokens at least
    const int64_t ctas = std::max<int64_t>((a.capacity + 2047) / 2048, (a.batch + 63) / 64);
    const int64_t cap = static_cast<int64_t>(device_sm_count());
    const PlanParams p = {a.cached, a.added, a.free_pages, a.table, a.q_start, a.kv_len, a.positions,
                          a.taken, a.slots, a.num_free, a.table_width, a.capacity, a.batch,
                          a.page_shift, ctx};
    return launch_kernel(plan_kernel, dim3(static_cast<unsigned>(std::min(ctas, cap))), dim3(kThreads),
                         smem, stream, 1, p);
}

cudaError_t launch_kv_append(const KvCache &c, const void *k, int64_t k_stride, const void *v,
                             int64_t v_stride, bool bf16, const int64_t *slots, int64_t n,
                             cudaStream_t stream, const LaunchCtx &ctx) {
    const int64_t threads = n * 2 * (static_cast<int64_t>(c.kv_heads) * c.head_dim / 4);
    const uintptr_t wide_bytes = bf16 ? 8 : 16;
    const bool wide = (reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) % wide_bytes == 0 &&
                      k_stride % 4 == 0 && v_stride % 4 == 0;
    const dim3 grid(grid_for(threads, 8));
    if (bf16)
        return launch_kernel(append_kernel<uint16_t>, grid, dim3(kThreads), 0, stream, 1, view(c),
                             static_cast<const uint16_t *>(k), k_stride,
                             static_cast<const uint16_t *>(v), v_stride, slots, n, c.head_dim,
                             static_cast<int>(wide), ctx);
    return launch_kernel(append_kernel<float>, grid, dim3(kThreads), 0, stream, 1, view(c),
                         static_cast<const float *>(k), k_stride, static_cast<const float *>(v),
                         v_stride, slots, n, c.head_dim, static_cast<int>(wide), ctx);
}

cudaError_t launch_kv_read(const KvCache &c, const int64_t *slots, int64_t n, float *k_out,
                           float *v_out, cudaStream_t stream, const LaunchCtx &ctx) {
    const int64_t threads = n * (static_cast<int64_t>(c.kv_heads) * c.head_dim / 4);
    const bool wide = ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 15) == 0;
    return launch_kernel(wide ? read_kernel<true> : read_kernel<false>, dim3(grid_for(threads, 8), 2), dim3(kThreads), 0, stream, 1,
                         view(c), slots, n, c.head_dim, k_out, v_out, ctx);
}

}  // namespace qmm
