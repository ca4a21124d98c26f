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
            // tokens without a row do not count: the others stand at their positions
            const int64_t here = had + min(tokens + now - had, p.capacity) - start[b];
            p.kv_len[b] = static_cast<int32_t>(min(here, static_cast<int64_t>(INT32_MAX)));
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
// Four lanes share a block of 32 values, eight each (two 16-byte loads of
// fp32, one of bf16); the extremes meet by shuffles, lanes 0 and 1 take the
// codes of lanes 2 and 3 as their high nibbles and write eight of the block's
// 16 bytes.  Bound by the bytes of the inputs; a decode step's few blocks are
// bound by latency.

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

// How a CTA's threads share tokens: `per` parts of eight values a token,
// several tokens at a time where they fit.  kAhead tokens per thread are
// loaded before the first is worked on: several where that still fills the
// GPU, else 1.  8191 tokens of 2 x 256 fp32, append and read: 20 us (79 MB,
// 3.9 TB/s; 27 with 1 and 1, 25 with 4 and 4, 21.4 where the registers allow
// only 4 and 3 CTAs an SM); 16 tokens: 3.6 us, 5.7 with several.
constexpr int kAppendMany = 2, kReadMany = 4;

struct Spread {
    int per, par, sub, at;
    __device__ explicit Spread(int parts) : per(parts) {
        par = max(1, kThreads / per);
        sub = threadIdx.x / per;
        at = threadIdx.x - sub * per;
        if (par == 1) {
            sub = 0;
            at = threadIdx.x;
        } else if (sub >= par) {
            at = per;  // threads that are left over
        }
    }
};

template <bool kWide>
__device__ __forceinline__ void load_eight(const float *p, float (&x)[8]) {
    if constexpr (kWide) {
        const float4 a = __ldcs(reinterpret_cast<const float4 *>(p)), b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = p[i];
    }
}
template <bool kWide>
__device__ __forceinline__ void load_eight(const uint16_t *p, float (&x)[8]) {
    if constexpr (kWide) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(static_cast<uint32_t>(p[i]) << 16);
    }
}

// Codes round(x / d) + 8 within 0..15 of eight values, a byte each, with the
// quotient rounded as IEEE division rounds and then to even.  x (1 / d) lies
// within 2^-22 of the quotient, relatively, so that it rounds to the same
// integer unless it is within 1e-5 of halfway between two (|x / d| < 16;
// larger ones are cut); only those are divided.
__device__ __forceinline__ void codes_of(const float (&x)[8], float d, uint32_t (&q)[2]) {
    constexpr float kOne = 12582912.0f;  // 1.5 2^23: here a unit is the last bit
    const float inv = __fdiv_rn(1.0f, d);
    float t[8], near = 0.5f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        t[i] = fminf(fmaxf(fmaf(x[i], inv, kOne), kOne - 8.0f), kOne + 7.0f);
        near = fminf(near, fabsf(fabsf(fmaf(x[i], inv, kOne - t[i])) - 0.5f));
    }
    if (near < 1e-5f) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            t[i] = kOne + fminf(fmaxf(rintf(__fdiv_rn(x[i], d)), -8.0f), 7.0f);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(t[4 * h + i] + 8.0f);
        q[h] = __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410);
    }
}

// kWide: rows of eight values are aligned to 16 bytes.  No pointer is
// __restrict__, here and in read: the compiler would take what they point to
// as constant for the kernel's lifetime, which begins before pdl_wait, while
// the kernel that writes it still runs.
template <typename T, bool kWide, int kAhead>
__global__ void __launch_bounds__(kThreads, 5) append_kernel(KvView c, const T *k, int64_t k_stride, const T *v,
                                                             int64_t v_stride, const int64_t *slots, int64_t n,
                                                             int dim, LaunchCtx ctx) {
    pdl_wait();
    pdl_launch_dependents();
    const int eights = c.kv_heads * dim / 8;  // of a token's keys, and of its values
    const Spread sp(2 * eights);
    // all of a warp's threads go through the loops: they shuffle
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * sp.par * kAhead; base < n;
         base += static_cast<int64_t>(gridDim.x) * sp.par * kAhead) {
        int64_t slot[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int64_t token = base + sp.sub + u * sp.par;
            slot[u] = token < n && sp.at < sp.per ? slots[token] : -1;
            if (slot[u] < -1 || slot[u] >= c.slots) {
                record_error(ctx, kDevErrIndex);
                slot[u] = -1;
            }
        }
        for (int i0 = 0; i0 < sp.per; i0 += kThreads) {
            const int i = i0 + sp.at;
            const bool here = i < sp.per;
            const int half = i >= eights, at = (i - half * eights) * 8;
            const T *src = (half ? v : k) + at;
            const int64_t stride = half ? v_stride : k_stride;
            float x[kAhead][8];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[u][j] = 0.0f;
                if (here && slot[u] >= 0) load_eight<kWide>(src + (base + sp.sub + u * sp.par) * stride, x[u]);
            }
            const int head = at / dim, in = at - head * dim, lane4 = threadIdx.x & 3;
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                float top = x[u][0], low = x[u][0], odd = 0.0f * x[u][0];  // 0 x is NaN for what a block cannot hold
#pragma unroll
                for (int j = 1; j < 8; ++j) {
                    top = fmaxf(top, x[u][j]);
                    low = fminf(low, x[u][j]);
                    odd = fmaf(0.0f, x[u][j], odd);
                }
#pragma unroll
                for (int o = 2; o > 0; o >>= 1) {
                    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                    low = fminf(low, __shfl_xor_sync(0xFFFFFFFFu, low, o));
                    odd += __shfl_xor_sync(0xFFFFFFFFu, odd, o);
                }
                const float e = top >= -low ? top : low;
                const __half dh = __float2half_rn(fminf(fmaxf(e * -0.125f, -65504.0f), 65504.0f));
                const float d = __half2float(dh);
                uint32_t q[2] = {0x08080808u, 0x08080808u};
                const bool finite = odd == 0.0f;
                if (finite && d != 0.0f) codes_of(x[u], d, q);
                const uint32_t high0 = __shfl_down_sync(0xFFFFFFFFu, q[0], 2, 4);
                const uint32_t high1 = __shfl_down_sync(0xFFFFFFFFu, q[1], 2, 4);
                if (!here || slot[u] < 0) continue;
                const int64_t row = cache_row(c, slot[u], head);
                if (lane4 < 2)
                    *reinterpret_cast<uint2 *>((half ? c.v_codes : c.k_codes) + row * (dim / 2) + (in / kQK) * 16 + lane4 * 8) =
                        make_uint2(q[0] | (high0 << 4), q[1] | (high1 << 4));
                if (lane4 == 0)
                    (half ? c.v_scales : c.k_scales)[row * (dim / kQK) + in / kQK] =
                        finite ? dh : __ushort_as_half(static_cast<unsigned short>(0x7FFF));
            }
        }
    }
}

// ---- read ----------------------------------------------------------------------
// Four lanes share a block: four bytes of codes each, which are four
// consecutive values of its first half and four of its second; keys and values
// as two halves of a token where both are wanted.  Bound by the bytes written.
template <bool kWide>
__device__ __forceinline__ void store_quad(float *dst, const float4 &y) {
    if constexpr (kWide) {
        *reinterpret_cast<float4 *>(dst) = y;
    } else {
        dst[0] = y.x;
        dst[1] = y.y;
        dst[2] = y.z;
        dst[3] = y.w;
    }
}

// (n - 8) f of four bytes: 2^23 + n - (2^23 + 8) is exact
__device__ __forceinline__ float4 values_of(uint32_t q, float f) {
    auto value = [&](uint32_t at) {
        return (__uint_as_float(__byte_perm(q, 0x4B000000u, 0x7440u | at)) - 8388616.0f) * f;
    };
    return make_float4(value(0), value(1), value(2), value(3));
}

template <bool kWide, int kAhead>
__global__ void __launch_bounds__(kThreads, 5) read_kernel(KvView c, const int64_t *slots, int64_t n, int dim,
                                                           float *k_out, float *v_out, LaunchCtx ctx) {
    pdl_wait();
    pdl_launch_dependents();
    const int eights = c.kv_heads * dim / 8;
    const int only = k_out ? (v_out ? -1 : 0) : 1;  // the half that is wanted, or both
    const Spread sp(only < 0 ? 2 * eights : eights);
    if (sp.at >= sp.per) return;
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
            const int half = only < 0 ? i >= eights : only, at = (only < 0 && half ? i - eights : i) * 8;
            const int head = at / dim, block = (at - head * dim) / kQK, quad = (at & 31) / 2;  // 4 times the lane
            const uint8_t *codes = half ? c.v_codes : c.k_codes;
            const __half *scales = half ? c.v_scales : c.k_scales;
            uint32_t w[kAhead];
            __half d[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                w[u] = 0x88888888u;  // zeros for slots that are not there
                d[u] = __ushort_as_half(0);
                if (slot[u] >= 0) {
                    const int64_t at_block = cache_row(c, slot[u], head) * (dim / kQK) + block;
                    w[u] = *reinterpret_cast<const uint32_t *>(codes + at_block * 16 + quad);
                    d[u] = scales[at_block];
                }
            }
            float *out = (half ? v_out : k_out) + (at & ~31) + quad;
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int64_t token = base + u * sp.par;
                if (token >= n) break;
                const float f = __half2float(d[u]);
                float *dst = out + token * eights * 8;
                store_quad<kWide>(dst, values_of(w[u] & 0x0F0F0F0Fu, f));
                store_quad<kWide>(dst + 16, values_of((w[u] >> 4) & 0x0F0F0F0Fu, f));
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

// CTAs for n tokens of `parts` parts each, `ahead` at a time, at most 32 per SM.
unsigned grid_for(int64_t n, int parts, int ahead) {
    const int64_t per_cta = static_cast<int64_t>(std::max(1, kThreads / parts)) * ahead;
    const int64_t cap = static_cast<int64_t>(device_sm_count()) * 32;
    return static_cast<unsigned>(std::min((n + per_cta - 1) / per_cta, cap));
}

// Whether CTAs of so many tokens a thread fill the GPU.
bool many(int64_t n, int parts, int ahead) {
    return grid_for(n, parts, ahead) >= static_cast<unsigned>(2 * device_sm_count());
}

template <typename T>
cudaError_t launch_append(const KvCache &c, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                          const int64_t *slots, int64_t n, cudaStream_t stream, const LaunchCtx &ctx) {
    constexpr int64_t values = 16 / sizeof(T);
    const bool wide = (reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) % 16 == 0 &&
                      k_stride % values == 0 && v_stride % values == 0;
    const int parts = c.kv_heads * c.head_dim / 4;
    const bool more = many(n, parts, kAppendMany);
    auto *kernel = wide ? (more ? append_kernel<T, true, kAppendMany> : append_kernel<T, true, 1>)
                        : (more ? append_kernel<T, false, kAppendMany> : append_kernel<T, false, 1>);
    return launch_kernel(kernel, dim3(grid_for(n, parts, more ? kAppendMany : 1)), dim3(kThreads), 0, stream, 1, view(c),
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
    const int parts = c.kv_heads * c.head_dim / 8 * (k_out && v_out ? 2 : 1);
    const bool more = many(n, parts, kReadMany);
    auto *kernel = wide ? (more ? read_kernel<true, kReadMany> : read_kernel<true, 1>)
                        : (more ? read_kernel<false, kReadMany> : read_kernel<false, 1>);
    return launch_kernel(kernel, dim3(grid_for(n, parts, more ? kReadMany : 1)), dim3(kThreads), 0, stream, 1, view(c),
                         slots, n, c.head_dim, k_out, v_out, ctx);
}

}  // namespace qmm
