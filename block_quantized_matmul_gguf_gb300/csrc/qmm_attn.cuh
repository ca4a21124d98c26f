// qmm_attn.cuh -- helpers shared by the attention kernels.
#pragma once

#include "qmm_internal.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace qmm {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// binary16 pair, lo in the low half: toward zero, or to nearest
__device__ __forceinline__ uint32_t pack_rz(float lo, float hi) {
    uint32_t r;
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack_rn(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
// the smaller and the larger of each half; NaN is passed over
__device__ __forceinline__ uint32_t hmin2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t hmax2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ float low_float(uint32_t v) {
    return __low2float(*reinterpret_cast<const __half2 *>(&v));
}
__device__ __forceinline__ float high_float(uint32_t v) {
    return __high2float(*reinterpret_cast<const __half2 *>(&v));
}

// 2^e for -126 <= e <= 127
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }
// floor(log2 x) of a positive normal x (-127 for zero and subnormals)
__device__ __forceinline__ int exponent(float x) { return static_cast<int>((__float_as_uint(x) >> 23) & 255u) - 127; }

__device__ __forceinline__ float load_value(const void *p, int64_t i, bool bf16) {
    if (bf16)
        return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(p)[i]) << 16);
    return static_cast<const float *>(p)[i];
}

__device__ __forceinline__ void store_value(void *p, int64_t i, bool bf16, float v) {
    if (bf16)
        static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
    else
        static_cast<float *>(p)[i] = v;
}

// The first key that position pos sees.
__device__ __forceinline__ int first_key(const AttnArgs &a, int pos) {
    return a.window && pos >= a.window ? pos - a.window + 1 : 0;
}

// A request's rows and keys, from device memory and within their arrays.
struct RequestRows {
    int row0, rows;  // first row of q, and rows that are there
    int len;         // keys, within the table
    int first;       // position of row row0 (may be negative)
    int bad;         // something had to be cut
};

__device__ __forceinline__ RequestRows request_rows(const AttnArgs &a, int page_shift, int b) {
    RequestRows r;
    const int s0 = a.q_start[b], s1 = a.q_start[b + 1], total = static_cast<int>(a.total_q);
    const int n = max(s1 - s0, 0), len = a.kv_len[b];
    r.row0 = min(max(s0, 0), total);
    r.rows = min(min(max(min(s1, total) - r.row0, 0), n), a.max_q);
    const int64_t room = min(a.table_width << page_shift, static_cast<int64_t>(INT32_MAX - 256));
    r.len = static_cast<int>(min(static_cast<int64_t>(max(len, 0)), room));
    r.first = max(len, 0) - n + (r.rows > 0 ? r.row0 - s0 : 0);  // rows cut in front keep their positions
    r.bad = s0 < 0 || s1 > total || s1 < s0 || n > a.max_q || len < 0 || len > room;
    return r;
}

// The power of two (as exponent) that brings a row of q with this largest
// value below 2^15, and the unit in which products with it count base-2
// scores: size * 2^(raise - up), a normal number.  size = |scale| log2(e).
__device__ __forceinline__ int query_raise(float big, float size) {
    return min(max(14 - exponent(big), max(-113, exponent(size) - 96)), 100);
}
__device__ __forceinline__ float score_unit(float size, int e) {
    return size == 0.0f ? 1.0f : fmaxf(size * pow2i(e / 2) * pow2i(e - e / 2), 1.17549435e-38f);
}

// Attention with the tensor cores' tiles (tcgen05), for bf16 outputs of
// prompts.  Whether it pays for these sizes: attn_tiles_pay.
bool attn_tiles_pay(const KvCache &cache, const AttnArgs &args);
size_t attn_tiles_workspace_bytes();
cudaError_t launch_attn_tiles(const KvCache &cache, const AttnArgs &args, cudaStream_t stream, const LaunchCtx &ctx);

}  // namespace qmm
