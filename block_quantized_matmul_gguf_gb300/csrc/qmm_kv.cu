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
    uint8_t *k_codes, *v_codes;
    __half *k_scales, *v_scales;
    int64_t slots;  // of the whole cache
    int page_shift, kv_heads;
};

// Row (page, head, place) of a slot, in rows of head_dim values.
__device__ __forceinline__ int64_t cache_row(const KvView &c, int64_t slot, int head) {
    const int64_t place = slot & ((int64_t(1) << c.page_shift) - 1);
    return ((((slot >> c.page_shift) * c.kv_heads) + head) << c.page_shift) + place;
}

// How a CTA's threads share tokens: `per` quads a token (a multiple of 32, so
// that a warp holds one token's), several tokens at a time where they fit.
// kAhead tokens per thread are loaded before the first is worked on: 4 where
// that still fills the GPU, else 1.  8191 tokens of 2 x 256 fp32, append and
// read: 29 us against 36 with 1; 16 tokens: 3.6 us against 5.7 with 4.
constexpr int kMany = 4;

struct Spread {
    int per, par, sub, at;
    __device__ explicit Spread(int quads) : per(quads) {
        par = max(1, kThreads / per);
        sub = threadIdx.x / per;
        at = threadIdx.x - sub * per;
        if (sub >= par) sub = -1;  // threads that are left over
    }
};

template <bool kWide>
__device__ __forceinline__ float4 load_quad(const float *p) {
    if constexpr (kWide) return __ldcs(reinterpret_cast<const float4 *>(p));
    return make_float4(p[0], p[1], p[2], p[3]);
}
template <bool kWide>
__device__ __forceinline__ float4 load_quad(const uint16_t *p) {
    uint32_t lo, hi;
    if constexpr (kWide) {
        const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(p));
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

// kWide: rows of quads are aligned to their size.
template <typename T, bool kWide, int kAhead>
__global__ void __launch_bounds__(kThreads) append_kernel(KvView c, const T *__restrict__ k,
                                                          int64_t k_stride,
                                                          const T *__restrict__ v,
                                                          int64_t v_stride,
                                                          const int64_t *__restrict__ slots,
                                                          int64_t n, int dim, LaunchCtx ctx) {
    pdl_wait();
    pdl_launch_dependents();
    const int quads = c.kv_heads * dim / 4;  // of a token's keys, and of its values
    const Spread sp(2 * quads);
    if (sp.sub < 0) return;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * sp.par * kAhead + sp.sub; base < n;
         base += static_cast<int64_t>(gridDim.x) * sp.par * kAhead) {
        int64_t slot[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int64_t token = base + u * sp.par;
            slot[u] = token < n ? slots[token] : -1;
            if (slot[u] < -1 || slot[u] >= c.slots) {
                record_error(ctx, kDevErrIndex);
                slot[u] = -1;
            }
        }
        for (int i = sp.at; i < sp.per; i += kThreads) {
            const int half = i >= quads, at = i - half * quads;
            const T *src = (half ? v : k) + at * 4;
            const int64_t stride = half ? v_stride : k_stride;
            float4 x[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                x[u] = slot[u] >= 0 ? load_quad<kWide>(src + (base + u * sp.par) * stride)
                                    : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            const int head = at * 4 / dim, block = (at * 4 - head * dim) / kQK, lane8 = threadIdx.x & 7;
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (slot[u] < 0) continue;  // the whole warp: one token
                float top = fmaxf(fmaxf(x[u].x, x[u].y), fmaxf(x[u].z, x[u].w));
                float low = fminf(fminf(x[u].x, x[u].y), fminf(x[u].z, x[u].w));
                // 0 * x is NaN for the values that a block cannot hold
                float odd = 0.0f * x[u].x + 0.0f * x[u].y + (0.0f * x[u].z + 0.0f * x[u].w);
#pragma unroll
                for (int o = 4; o > 0; o >>= 1) {
                    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                    low = fminf(low, __shfl_xor_sync(0xFFFFFFFFu, low, o));
                    odd += __shfl_xor_sync(0xFFFFFFFFu, odd, o);
                }
                const float e = top >= -low ? top : low;
                const __half dh = __float2half_rn(fminf(fmaxf(e * -0.125f, -65504.0f), 65504.0f));
                const float d = __half2float(dh);
                uint32_t q = 0x08080808u;
                const bool finite = odd == 0.0f;
                if (finite && d != 0.0f)
                    q = code_of(x[u].x, d) | (code_of(x[u].y, d) << 8) | (code_of(x[u].z, d) << 16) |
                        (code_of(x[u].w, d) << 24);
                const uint32_t high = __shfl_down_sync(0xFFFFFFFFu, q, 4, 8);
                const int64_t row = cache_row(c, slot[u], head);
                if (lane8 < 4)
                    *reinterpret_cast<uint32_t *>((half ? c.v_codes : c.k_codes) + row * (dim / 2) + block * 16 + lane8 * 4) =
                        q | (high << 4);
                if (lane8 == 0)
                    (half ? c.v_scales : c.k_scales)[row * (dim / kQK) + block] =
                        finite ? dh : __ushort_as_half(static_cast<unsigned short>(0x7FFF));
            }
        }
    }
}

// ---- read ----------------------------------------------------------------------
// Eight lanes share a block, four consecutive values each (as dequant); keys
// and values as two halves of a token where both are wanted.
template <bool kWide, int kAhead>
__global__ void __launch_bounds__(kThreads) read_kernel(KvView c, const int64_t *__restrict__ slots,
                                                        int64_t n, int dim, float *__restrict__ k_out,
                                                        float *__restrict__ v_out, LaunchCtx ctx) {
    pdl_wait();
    pdl_launch_dependents();
    const int quads = c.kv_heads * dim / 4;
    const int only = k_out ? (v_out ? -1 : 0) : 1;  // the half that is wanted, or both
    const Spread sp(only < 0 ? 2 * quads : quads);
    if (sp.sub < 0) return;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * sp.par * kAhead + sp.sub; base < n;
         base += static_cast<int64_t>(gridDim.x) * sp.par * kAhead) {
        int64_t slot[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int64_t token = base + u * sp.par;
            slot[u] = token < n ? slots[token] : -1;
            if (slot[u] < -1 || slot[u] >= c.slots) {
                record_error(ctx, kDevErrIndex);
                slot[u] = -1;
            }
        }
        for (int i = sp.at; i < sp.per; i += kThreads) {
            const int half = only < 0 ? i >= quads : only, at = (only < 0 && half ? i - quads : i) * 4;
            const int head = at / dim, in = at - head * dim;
            uint32_t w[kAhead];
            __half d[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                w[u] = 0x88888888u;  // zeros for slots that are not there
                d[u] = __ushort_as_half(0);
                if (slot[u] >= 0) {
                    const int64_t row = cache_row(c, slot[u], head);
                    w[u] = *reinterpret_cast<const uint32_t *>((half ? c.v_codes : c.k_codes) + row * (dim / 2) + (in / kQK) * 16 + (in & 15));
                    d[u] = (half ? c.v_scales : c.k_scales)[row * (dim / kQK) + in / kQK];
                }
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int64_t token = base + u * sp.par;
                if (token >= n) break;
                const uint32_t q = w[u] >> ((in & 16) ? 4 : 0);
                const float f = __half2float(d[u]);
                float4 y;
                y.x = (static_cast<float>(q & 15u) - 8.0f) * f;
                y.y = (static_cast<float>((q >> 8) & 15u) - 8.0f) * f;
                y.z = (static_cast<float>((q >> 16) & 15u) - 8.0f) * f;
                y.w = (static_cast<float>((q >> 24) & 15u) - 8.0f) * f;
                float *dst = (half ? v_out : k_out) + token * quads * 4 + at;
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
    }
}

KvView view(const KvCache &c) {
    KvView v;
    v.k_codes = static_cast<uint8_t *>(c.k_codes);
    v.v_codes = static_cast<uint8_t *>(c.v_codes);
    v.k_scales = static_cast<__half *>(c.k_scales);
    v.v_scales = static_cast<__half *>(c.v_scales);
    v.slots = c.num_pages << c.page_shift;
    v.page_shift = c.page_shift;
    v.kv_heads = c.kv_heads;
    return v;
}

// CTAs for n tokens of `quads` quads each, `ahead` at a time, at most 32 per SM.
unsigned grid_for(int64_t n, int quads, int ahead) {
    const int64_t per_cta = static_cast<int64_t>(std::max(1, kThreads / quads)) * ahead;
    const int64_t cap = static_cast<int64_t>(device_sm_count()) * 32;
    return static_cast<unsigned>(std::min((n + per_cta - 1) / per_cta, cap));
}

// Whether CTAs of kMany tokens fill the GPU.
bool many(int64_t n, int quads) {
    return grid_for(n, quads, kMany) >= static_cast<unsigned>(2 * device_sm_count());
}

template <typename T>
cudaError_t launch_append(const KvCache &c, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                          const int64_t *slots, int64_t n, cudaStream_t stream, const LaunchCtx &ctx) {
    constexpr uintptr_t quad = 4 * sizeof(T);
    const bool wide = (reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) % quad == 0 &&
                      k_stride % 4 == 0 && v_stride % 4 == 0;
    const int quads = c.kv_heads * c.head_dim / 2;
    const bool more = many(n, quads);
    auto *kernel = wide ? (more ? append_kernel<T, true, kMany> : append_kernel<T, true, 1>)
                        : (more ? append_kernel<T, false, kMany> : append_kernel<T, false, 1>);
    return launch_kernel(kernel, dim3(grid_for(n, quads, more ? kMany : 1)), dim3(kThreads), 0, stream, 1, view(c),
                         static_cast<const T *>(k), k_stride, static_cast<const T *>(v), v_stride, slots, n,
                         c.head_dim, ctx);
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
    return bf16 ? launch_append<uint16_t>(c, k, k_stride, v, v_stride, slots, n, stream, ctx)
                : launch_append<float>(c, k, k_stride, v, v_stride, slots, n, stream, ctx);
}

cudaError_t launch_kv_read(const KvCache &c, const int64_t *slots, int64_t n, float *k_out,
                           float *v_out, cudaStream_t stream, const LaunchCtx &ctx) {
    const bool wide = ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 15) == 0;
    const int quads = c.kv_heads * c.head_dim / 4 * (k_out && v_out ? 2 : 1);
    const bool more = many(n, quads);
    auto *kernel = wide ? (more ? read_kernel<true, kMany> : read_kernel<true, 1>)
                        : (more ? read_kernel<false, kMany> : read_kernel<false, 1>);
    return launch_kernel(kernel, dim3(grid_for(n, quads, more ? kMany : 1)), dim3(kThreads), 0, stream, 1, view(c),
                         slots, n, c.head_dim, k_out, v_out, ctx);
}

}  // namespace qmm
