// qmm_experts.cuh -- the experts' Q4_0 products (include/qmm.h,
// qmm_experts_geglu_q4_0 and qmm_experts_down_q4_0): the streaming form, for
// few rows an expert and for fp32 outputs.
//
// Mathematics.  With codes n (0..15) and scales d of 32-weight blocks b,
//   y[i] = sum_b d_b * sum_j (n_bj - 8) x_bj
// for the rows x of an expert's pairs.  The integers are exact in binary16 and bf16, so
// the inner sums run on mma.sync m16n8k16 with 16 rows of weights as one
// operand, taken from the 4-bit codes in registers, and 8 pairs' x as the other;
// the scales join in fp32.
//
// Precision.  A bf16 x enters as it is (PARTS 1).  An fp32 x enters in two binary16
// parts (PARTS 2), scaled by a power of two per row and 256 values so that the largest
// lies in [2^14, 2^15): 22 bits, down to 2^-39 of that largest.  They are two products into
// one sum, or, for groups of eight pairs, other columns of one product (`split`), whose
// eight columns then are four pairs, so that a group has two.  Each part is then a
// sum of its own and both meet at the end, however full the group is: a pair's bits
// do not depend on the others (16 tokens of 8 of 64 experts of 1024 x 2048: 43 us).
// The codes are made n - 8 before the products: left as the subnormal numbers that a
// word holds they save two instructions a pair, but the tensor cores' sums of
// subnormal operands keep some 18 bits only.
//
// Work.  An item is 64 rows of weights (32 gate and the same 32 up rows for
// GeGLU) of one expert against one group of 8 NB of its pairs.  A CTA of up to 8
// warps, one an SM, walks through its own run of items: RW items at a time, each
// by KW warps that take every KW-th 256 values of K and add their sums in shared
// memory in a fixed order.  The group's x lies in shared memory as the
// instruction wants it, made once while the items stay with the group, or with
// rows of the same token.  Each warp's weights arrive through its own two stages of
// 64 rows x 144 bytes, so that the eight rows that a quarter of a load touches lie
// in different banks: by TMA where K is a multiple of 256, by cp.async otherwise.
#pragma once

#include "qmm_tc.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

namespace qmm {
namespace experts {

constexpr int kMaxWarps = 8;
constexpr int kStages = 2;
constexpr int kChunk = 256;   // K values of a stage
constexpr int kTiles = 4;     // of 16 weight rows, of an item
constexpr int kRows = 16 * kTiles;

constexpr int kMostUnits = (1 << 30) - 1;  // where sums stop: above those of any plan, and twice it fits

struct StreamParams {
    ExpertsPlan plan;
    const uint8_t *w[2];  // GeGLU: gate and up; down: w[0]
    const void *x;
    int64_t x_stride;     // elements
    void *out;            // GeGLU: h, by the pairs' order; down: fp32 [pairs], by the pair
    int64_t out_stride;   // elements
    int64_t n, k;
    int64_t row_bytes;    // of weights
    int64_t matrix_bytes; // of an expert
    int64_t w_bytes;      // of all
    int chunks;           // of K
    int blocks;           // of K
    int rw, kw;           // items at a time, warps an item
    int row_groups;       // items of rw * rows
    int x_panel;          // chunks of x that shared memory holds
    uint32_t magic;       // 1024, 1024 in binary16, or 16, 16 in bf16, in a register
    bool x_bf16, out_bf16, x_wide;
    LaunchCtx ctx;
};

__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float low_half(uint32_t v) { return __low2float(*reinterpret_cast<const __half2 *>(&v)); }
__device__ __forceinline__ float high_half(uint32_t v) { return __high2float(*reinterpret_cast<const __half2 *>(&v)); }

// d = a b + c, a 16 x 16 (row), b 16 x 8 (column), binary16 or bf16, fp32 sums
template <bool BF16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 bytes, of which the first `bytes` are read and the others zeros
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void barrier(int id, int threads) {
    asm volatile("barrier.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// How a group of 8 NB pairs lies in the products: blocks of eight columns, and the parts
// of x that are products of their own; split: columns 0 .. 3 are four pairs' large parts, 4 .. 7 their small ones.
template <int PARTS, int NB>
struct Columns {
    static constexpr bool split = PARTS == 2 && NB == 1;
    static constexpr int blocks = split ? 2 : NB, parts = split ? 1 : PARTS;
    static constexpr int pairs = split ? 4 : 8;    // of a block
    static constexpr int lanes = split ? 16 : 32;  // of a warp that hold sums of their own
};

// Shared memory, from its start: rings, x, its scales, partial sums, rows.
template <int PARTS, int NB, bool ALIGNED>
struct StreamLayout {
    static constexpr int pitch = ALIGNED ? 144 : 176;  // bytes of a row's window in a stage
    static constexpr int stage = kRows * pitch;
    static constexpr int x_block = NB * PARTS * 512;   // bytes of 32 values of K
    __host__ __device__ static int x(int warps) { return warps * kStages * stage; }
    __host__ __device__ static int scale(int warps, int panel) { return x(warps) + panel * 8 * x_block; }
    __host__ __device__ static int part(int warps, int panel) { return scale(warps, panel) + panel * Columns<PARTS, NB>::blocks * 32; }
    __host__ __device__ static int rows(int warps, int panel) { return part(warps, panel) + warps * NB * kTiles * 512; }
    __host__ __device__ static int total(int warps, int panel) { return rows(warps, panel) + 2 * 8 * NB * 4 + 64; }
};

// A place in a CTA's run of items.
struct Place {
    int left;  // items of the run from here on
    int expert, group, row_group;
    int start, count;  // of the expert's pairs
};

// The pairs of an expert, bounded.
__device__ __forceinline__ void expert_range(const StreamParams &p, int e, int &start, int &count) {
    const int64_t pairs = p.plan.pairs_total;
    const int64_t a = p.plan.expert_start[e], b = p.plan.expert_start[e + 1];
    if (a < 0 || b < a || b > pairs) {
        record_error(p.ctx, kDevErrIndex);
        start = 0;
        count = 0;
        return;
    }
    start = static_cast<int>(a);
    count = static_cast<int>(b - a);
}

template <int NB>
__device__ __forceinline__ void advance(const StreamParams &p, Place &at) {
    if (--at.left <= 0) return;
    if (++at.row_group < p.row_groups) return;
    at.row_group = 0;
    ++at.group;
    while (at.group * 8 * NB >= at.count) {
        if (++at.expert >= p.plan.experts) {  // cannot be: the run ends before
            at.left = 0;
            return;
        }
        at.group = 0;
        expert_range(p, at.expert, at.start, at.count);
    }
}

// An item's rows x one chunk of weights into a stage of this warp's ring: by TMA
// boxes where rows allow it, else as the windows of 16-byte pieces that hold them.
template <bool GEGLU>
__device__ __forceinline__ void load_boxes(const StreamParams &p, const CUtensorMap *w0, const CUtensorMap *w1, uint32_t stage,
                                           uint32_t bar, int expert, int64_t row0, int chunk) {
    const int row = static_cast<int>(expert * p.n + row0);  // rows behind the expert's are not stored
    mbar_expect_tx_addr(bar, kRows * 144);
    tma_load_2d(stage, w0, chunk * 144, row, bar);
    if constexpr (GEGLU) tma_load_2d(stage + kRows / 2 * 144, w1, chunk * 144, row, bar);
}
// Ten pieces a row, 32 rows in ten steps, which repeat: a row's skew does, as the bytes
// of 32 rows are a multiple of 16.
struct Windows {
    int64_t base = -1, first;  // of the item's rows, and down to 16 bytes
    int at[10];                // the lane's pieces from there
};
template <bool GEGLU>
__device__ __forceinline__ void load_windows(const StreamParams &p, Windows &win, uint32_t stage, int expert, int64_t row0, int chunk,
                                             int lane) {
    constexpr int pitch = 176, pieces = 10;
    const int64_t base = expert * p.matrix_bytes + row0 * p.row_bytes;
    auto piece = [&](int i) {
        const int at32 = i * 32 + lane;
        return ((base + at32 / pieces * p.row_bytes) & ~int64_t(15)) - (base & ~int64_t(15)) + at32 % pieces * 16;
    };
    auto place = [&](int i) { return (i * 32 + lane) / pieces * pitch + (i * 32 + lane) % pieces * 16; };
    if (base != win.base) {
        win.base = base;
        win.first = base & ~int64_t(15);
#pragma unroll
        for (int i = 0; i < pieces; ++i) win.at[i] = static_cast<int>(piece(i));
    }
#pragma unroll 1
    for (int rows32 = 0; rows32 < kRows / 32; ++rows32) {  // rows behind the expert's are not stored
        const uint8_t *w = p.w[GEGLU ? rows32 : 0];
        const int64_t from = win.first + (GEGLU ? 0 : rows32) * 32 * p.row_bytes + chunk * 144;
        const uint32_t to = stage + rows32 * 32 * pitch;
        if (from + 32 * p.row_bytes + pitch <= p.w_bytes) {  // windows end below 31 rows + 176 bytes
#pragma unroll
            for (int i = 0; i < pieces; ++i) copy16(to + place(i), w + from + win.at[i], 16);
        } else {
#pragma unroll 1
            for (int i = 0; i < pieces; ++i) {
                const int64_t at = from + piece(i), left = p.w_bytes - at;
                copy16(to + place(i), w + (left > 0 ? at : 0), left >= 16 ? 16u : left > 0 ? static_cast<uint32_t>(left) : 0u);
            }
        }
    }
}

__device__ __forceinline__ float4 load_four(const float *p, bool wide) {
    if (wide) return *reinterpret_cast<const float4 *>(p);
    return make_float4(p[0], p[1], p[2], p[3]);
}
__device__ __forceinline__ uint2 load_four(const uint16_t *p, bool wide) {
    if (wide) return *reinterpret_cast<const uint2 *>(p);
    return make_uint2(p[0] | static_cast<uint32_t>(p[1]) << 16, p[2] | static_cast<uint32_t>(p[3]) << 16);
}

// One chunk of x as the products' operand, eight columns of it: lane (g, t) makes
// column g's values 4t..4t+3 and 16+4t..16+4t+3 of each block, in the order that
// the codes of a word have.  bf16 values stay as they are.
template <int NB>
__device__ __noinline__ void stage_x(const StreamParams &p, char *xs, float *, const uint16_t *row, int chunk, int nb, int lane) {
    const int t = lane & 3;
    const int blocks = min(8, p.blocks - chunk * 8);
#pragma unroll
    for (int b = 0; b < 8; ++b) {
        uint2 v[2] = {};
        if (row && b < blocks)
#pragma unroll
            for (int h = 0; h < 2; ++h) v[h] = load_four(row + chunk * kChunk + b * 32 + h * 16 + 4 * t, p.x_wide);
        reinterpret_cast<uint4 *>(xs + ((chunk * 8 + b) * NB + nb) * 512)[lane] =
            make_uint4(__byte_perm(v[0].x, v[0].y, 0x5410), __byte_perm(v[0].x, v[0].y, 0x7632),
                       __byte_perm(v[1].x, v[1].y, 0x5410), __byte_perm(v[1].x, v[1].y, 0x7632));
    }
}
template <int NB>
__device__ __noinline__ void stage_x(const StreamParams &p, char *xs, float *scale, const float *row, int chunk, int nb, int lane) {
    constexpr int PARTS = 2;
    using C = Columns<PARTS, NB>;
    const int t = lane & 3, g = lane >> 2;
    const int blocks = min(8, p.blocks - chunk * 8);
    float4 v[8][2];
    float top = 0.0f;
#pragma unroll
    for (int b = 0; b < 8; ++b) {
        v[b][0] = v[b][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (row && b < blocks) {
            v[b][0] = load_four(row + chunk * kChunk + b * 32 + 4 * t, p.x_wide);
            v[b][1] = load_four(row + chunk * kChunk + b * 32 + 16 + 4 * t, p.x_wide);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
            top = fmaxf(fmaxf(fmaxf(top, fabsf(v[b][h].x)), fabsf(v[b][h].y)), fmaxf(fabsf(v[b][h].z), fabsf(v[b][h].w)));
    }
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    // top 2^f in [2^14, 2^15); both powers normal (a smaller top stays smaller)
    const int e = min(max(static_cast<int>(__float_as_uint(top) >> 23), 15), 254);
    const float f = __uint_as_float(static_cast<uint32_t>(268 - e) << 23);
    if (t == 0) scale[(chunk * C::blocks + nb) * 8 + g] = __uint_as_float(static_cast<uint32_t>(e - 14) << 23);
#pragma unroll
    for (int b = 0; b < 8; ++b) {
        uint32_t part[PARTS][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float y[4] = {v[b][h].x * f, v[b][h].z * f, v[b][h].y * f, v[b][h].w * f};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t hi = pack_half(y[2 * i], y[2 * i + 1]);
                part[0][2 * h + i] = hi;
                part[1][2 * h + i] = pack_half(y[2 * i] - low_half(hi), y[2 * i + 1] - high_half(hi));
            }
        }
        char *to = xs + ((chunk * 8 + b) * C::blocks + nb) * C::parts * 512;
        if constexpr (C::split) {
            const bool low = g >= 4;
            reinterpret_cast<uint4 *>(to)[lane] = make_uint4(low ? part[1][0] : part[0][0], low ? part[1][1] : part[0][1],
                                                             low ? part[1][2] : part[0][2], low ? part[1][3] : part[0][3]);
        } else {
#pragma unroll
            for (int q = 0; q < PARTS; ++q)
                reinterpret_cast<uint4 *>(to + q * 512)[lane] = make_uint4(part[q][0], part[q][1], part[q][2], part[q][3]);
        }
    }
}

// A warp's products of one stage: kTiles tiles of 16 rows against the first USED
// of NB blocks of eight columns.  skew: bytes by which the lane's rows (g, g + 8 of each tile, which
// repeat after two) begin behind their windows.
template <bool BF16, int PARTS, int NB, int USED, bool ALIGNED>
__device__ __forceinline__ void stage_products(const char *stage, const char *xs, const float *scale, int blocks,
                                               const int (&skew)[2][2], uint32_t magic, int lane,
                                               float (&total)[kTiles][NB][4]) {
    constexpr int pitch = ALIGNED ? 144 : 176;
    const int t = lane & 3, g = lane >> 2;
    float acc[kTiles][USED][4];
#pragma unroll
    for (int r = 0; r < kTiles; ++r)
#pragma unroll
        for (int n = 0; n < USED; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[r][n][i] = BF16 ? total[r][n][i] : 0.0f;
    auto block = [&](int b, const uint32_t (&q)[kTiles][2], const float (&d)[kTiles][2]) {
        uint32_t x[USED][PARTS][4];
#pragma unroll
        for (int n = 0; n < USED; ++n) {
#pragma unroll
            for (int s = 0; s < PARTS; ++s) {
                const uint4 v = reinterpret_cast<const uint4 *>(xs + ((b * NB + n) * PARTS + s) * 512)[lane];
                x[n][s][0] = v.x, x[n][s][1] = v.y, x[n][s][2] = v.z, x[n][s][3] = v.w;
            }
        }
        // the products of the tiles take turns: each waits for the one before it of
        // its own sum
        uint32_t a[kTiles][8];
#pragma unroll
        for (int r = 0; r < kTiles; ++r) {
            const uint32_t u = q[r][0], v = q[r][1];
            if constexpr (BF16) {  // 16 + n, n in the place of 16's upper mantissa bits, - 24
                auto codes = [&](uint32_t w) { return add_bf16x2((w & 0x00780078u) | magic, 0xC1C0C1C0u); };
                a[r][0] = codes(u << 3), a[r][1] = codes(v << 3), a[r][2] = codes(u >> 5), a[r][3] = codes(v >> 5);
                a[r][4] = codes(u >> 1), a[r][5] = codes(v >> 1), a[r][6] = codes(u >> 9), a[r][7] = codes(v >> 9);
            } else {
                const uint32_t u8 = u >> 8, v8 = v >> 8;
                a[r][0] = hadd2((u & 0x000F000Fu) | magic, 0xE408E408u);  // - 1032
                a[r][1] = hadd2((v & 0x000F000Fu) | magic, 0xE408E408u);
                a[r][2] = hadd2((u8 & 0x000F000Fu) | magic, 0xE408E408u);
                a[r][3] = hadd2((v8 & 0x000F000Fu) | magic, 0xE408E408u);
                a[r][4] = hfma2((u & 0x00F000F0u) | magic, 0x2C002C00u, 0xD480D480u);  // / 16 - 72
                a[r][5] = hfma2((v & 0x00F000F0u) | magic, 0x2C002C00u, 0xD480D480u);
                a[r][6] = hfma2((u8 & 0x00F000F0u) | magic, 0x2C002C00u, 0xD480D480u);
                a[r][7] = hfma2((v8 & 0x00F000F0u) | magic, 0x2C002C00u, 0xD480D480u);
            }
        }
#pragma unroll
        for (int n = 0; n < USED; ++n) {
            float z[kTiles][4];
#pragma unroll
            for (int r = 0; r < kTiles; ++r) z[r][0] = z[r][1] = z[r][2] = z[r][3] = 0.0f;
#pragma unroll
            for (int s = PARTS - 1; s >= 0; --s) {  // the small part first
#pragma unroll
                for (int r = 0; r < kTiles; ++r)
                    mma<BF16>(z[r], a[r][0], a[r][1], a[r][2], a[r][3], x[n][s][0], x[n][s][1]);
#pragma unroll
                for (int r = 0; r < kTiles; ++r)
                    mma<BF16>(z[r], a[r][4], a[r][5], a[r][6], a[r][7], x[n][s][2], x[n][s][3]);
            }
#pragma unroll
            for (int r = 0; r < kTiles; ++r) {
                acc[r][n][0] = fmaf(d[r][0], z[r][0], acc[r][n][0]);
                acc[r][n][1] = fmaf(d[r][0], z[r][1], acc[r][n][1]);
                acc[r][n][2] = fmaf(d[r][1], z[r][2], acc[r][n][2]);
                acc[r][n][3] = fmaf(d[r][1], z[r][3], acc[r][n][3]);
            }
        }
    };
    if constexpr (ALIGNED) {
        // two blocks are nine words: the first block's codes begin in the
        // middle of a word, the second's at one
#pragma unroll (USED > 1 ? 1 : 2)
        for (int j = 0; j < 4; ++j) {
            uint32_t q0[kTiles][2], q1[kTiles][2];
            float d0[kTiles][2], d1[kTiles][2];
#pragma unroll
            for (int r = 0; r < kTiles; ++r)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const char *row = stage + (r * 16 + h * 8 + g) * pitch + 36 * j;
                    const uint32_t *w = reinterpret_cast<const uint32_t *>(row) + t;
                    q0[r][h] = __byte_perm(w[0], w[1], 0x5432);
                    q1[r][h] = w[5];
                    d0[r][h] = half_bits_to_float(*reinterpret_cast<const uint16_t *>(row));
                    d1[r][h] = half_bits_to_float(*reinterpret_cast<const uint16_t *>(row + 18));
                }
            block(2 * j, q0, d0);
            block(2 * j + 1, q1, d1);
        }
    } else {
        // the same behind each row's skew; an odd number of blocks ends with one of scale 0
#pragma unroll (USED > 1 ? 1 : 2)
        for (int j = 0; 2 * j < blocks; ++j) {
            uint32_t q0[kTiles][2], q1[kTiles][2];
            float d0[kTiles][2], d1[kTiles][2];
            const bool both = 2 * j + 1 < blocks;
#pragma unroll
            for (int r = 0; r < kTiles; ++r)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int at = skew[r & 1][h];  // repeats after 32 rows
                    const char *row = stage + (r * 16 + h * 8 + g) * pitch + 36 * j;
                    const uint32_t *w = reinterpret_cast<const uint32_t *>(row + (at & ~3)) + t;
                    q0[r][h] = __byte_perm(w[0], w[1], at & 2 ? 0x7654 : 0x5432);
                    q1[r][h] = __byte_perm(w[5], w[6], at & 2 ? 0x5432 : 0x3210);
                    d0[r][h] = half_bits_to_float(*reinterpret_cast<const uint16_t *>(row + at));
                    d1[r][h] = both ? half_bits_to_float(*reinterpret_cast<const uint16_t *>(row + at + 18)) : 0.0f;
                }
            block(2 * j, q0, d0);
            block(2 * j + 1, q1, d1);
        }
    }
#pragma unroll
    for (int n = 0; n < USED; ++n) {
        const float2 s = BF16 ? float2{} : *reinterpret_cast<const float2 *>(scale + n * 8 + 2 * t);
#pragma unroll
        for (int r = 0; r < kTiles; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                total[r][n][i] = BF16 ? acc[r][n][i] : fmaf(acc[r][n][i], i & 1 ? s.y : s.x, total[r][n][i]);
    }
}

// gelu(z) = z / 2 (1 + tanh(a)) = z / (1 + exp(-2a))
__device__ __forceinline__ float gelu(float z) {
    const float a = 0.7978845608028654f * fmaf(0.044715f * z, z * z, z);
    return z / (1.0f + expf(-2.0f * a));
}

__device__ __forceinline__ void put(void *out, int64_t at, bool bf16, float v) {
    if (bf16)
        static_cast<__nv_bfloat16 *>(out)[at] = __float2bfloat16_rn(v);
    else
        static_cast<float *>(out)[at] = v;
}

template <int PARTS, int NB, bool GEGLU, bool ALIGNED>
__global__ void __launch_bounds__(kMaxWarps * 32, 1) stream_kernel(const __grid_constant__ CUtensorMap w0,
                                                                   const __grid_constant__ CUtensorMap w1,
                                                                   const __grid_constant__ StreamParams p) {
    using L = StreamLayout<PARTS, NB, ALIGNED>;
    using C = Columns<PARTS, NB>;
    extern __shared__ __align__(128) char smem[];
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = lane & 3, g = lane >> 2;
    const int rw = warp / p.kw, kw = warp - rw * p.kw;  // item among those at a time, part of K
    char *xs = smem + L::x(warps);
    float *scale = reinterpret_cast<float *>(smem + L::scale(warps, p.x_panel));
    float *part = reinterpret_cast<float *>(smem + L::part(warps, p.x_panel));
    int *src = reinterpret_cast<int *>(smem + L::rows(warps, p.x_panel));  // [8 NB] rows of x, -1 where there is none
    int *dst = src + 8 * NB;                                              // [8 NB] rows of out
    int *found = dst + 8 * NB;                                            // the run's first place

    pdl_wait();
    pdl_launch_dependents();

    // The run: units (expert, group of pairs) x row groups, cut equally.
    {
        __shared__ int32_t sum[kMaxWarps];
        const int threads = blockDim.x;
        const int per = (p.plan.experts + threads - 1) / threads;
        const int e0 = min(p.plan.experts, static_cast<int>(threadIdx.x) * per), e1 = min(p.plan.experts, e0 + per);
        int mine = 0;
        for (int e = e0; e < e1; ++e) {
            int start, count;
            expert_range(p, e, start, count);
            mine += (count + 8 * NB - 1) / (8 * NB);
        }
        int s = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, s, o);
            if (lane >= o) s = min(s + u, kMostUnits);
        }
        if (lane == 31) sum[warp] = s;
        __syncthreads();
        int ahead = s - mine, all = 0;
        for (int w = 0; w < warps; ++w) {
            if (w < warp) ahead = min(ahead + sum[w], kMostUnits);
            all = min(all + sum[w], kMostUnits);
        }
        // a plan whose experts claim more than its pairs is not worked: sums stay exact
        if (all > p.plan.pairs_total / (8 * NB) + p.plan.experts) {
            if (threadIdx.x == 0) record_error(p.ctx, kDevErrIndex);
            return;
        }
        const int64_t items = static_cast<int64_t>(all) * p.row_groups;
        const int64_t from = items * blockIdx.x / gridDim.x, to = items * (blockIdx.x + 1) / gridDim.x;
        if (from == to) return;
        const int unit = static_cast<int>(from / p.row_groups);
        if (unit >= ahead && unit < ahead + mine) {  // one thread of the CTA
            for (int e = e0; e < e1; ++e) {
                int start, count;
                expert_range(p, e, start, count);
                const int units = (count + 8 * NB - 1) / (8 * NB);
                if (unit < ahead + units) {
                    found[0] = e;
                    found[1] = unit - ahead;
                    found[2] = start;
                    found[3] = count;
                    break;
                }
                ahead += units;
            }
            found[4] = static_cast<int>(from - static_cast<int64_t>(unit) * p.row_groups);
            found[5] = static_cast<int>(to - from);
        }
        __syncthreads();
    }
    Place at;
    at.expert = found[0];
    at.group = found[1];
    at.start = found[2];
    at.count = found[3];
    at.row_group = found[4];
    at.left = found[5];

    constexpr int kItemRows = GEGLU ? kRows / 2 : kRows;
    constexpr int kPairs = GEGLU ? kTiles / 2 : kTiles;  // tiles of out
    const uint32_t ring = smem_addr(smem) + warp * kStages * L::stage;
    const char *ring_ptr = smem + warp * kStages * L::stage;

    // A chunk of weights is on its way while the one before is worked on, through the
    // items.  A wait that runs out leaves the rest undone, but not the barriers.
    __shared__ alignas(8) uint64_t bars[kMaxWarps][kStages];
    bool ok = true;
    if constexpr (ALIGNED) {
        if (lane < kStages) mbar_init(&bars[warp][lane], 1);
        fence_mbar_init();
        __syncwarp();
    }
    Windows windows;
    auto load = [&](const Place &from, int chunk, int turn) {
        const int slot = turn & (kStages - 1);
        const int64_t row0 = (static_cast<int64_t>(from.row_group) * p.rw + rw) * kItemRows;
        const bool there = from.left > 0 && row0 < p.n && ok;
        if constexpr (ALIGNED) {
            if (there && lane == 0)
                load_boxes<GEGLU>(p, &w0, &w1, ring + slot * L::stage, smem_addr(&bars[warp][slot]), from.expert, row0, chunk);
        } else {
            if (there) load_windows<GEGLU>(p, windows, ring + slot * L::stage, from.expert, row0, chunk, lane);
            copy_commit();
        }
    };
    uint32_t parity = 0;  // of each stage's barrier, a bit
    load(at, kw, 0);

    int done = 0;
    int held_expert = -1, held_group = -1, held_panel = -1;
    const int panels = (p.chunks + p.x_panel - 1) / p.x_panel;
    while (at.left > 0) {
        Place next = at;
        const int64_t row0 = (static_cast<int64_t>(at.row_group) * p.rw + rw) * kItemRows;
        const bool there = row0 < p.n;
        const int first = at.start + at.group * 8 * NB;              // of the pairs
        const int cols = min(8 * NB, at.count - at.group * 8 * NB);  // of them here
        const int used = (cols + C::pairs - 1) / C::pairs;           // blocks of columns
        float total[kTiles][C::blocks][4];
#pragma unroll
        for (int r = 0; r < kTiles; ++r)
#pragma unroll
            for (int n = 0; n < C::blocks; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) total[r][n][i] = 0.0f;
        int skew[2][2] = {};
        if constexpr (!ALIGNED) {
            const int64_t base = at.expert * p.matrix_bytes + row0 * p.row_bytes;
#pragma unroll
            for (int i = 0; i < 4; ++i) skew[i >> 1][i & 1] = static_cast<int>(base + (i * 8 + g) * p.row_bytes) & 15;
        }
        for (int panel = 0; panel < panels; ++panel) {
            const int c0 = panel * p.x_panel, c1 = min(p.chunks, c0 + p.x_panel);
            if (at.expert != held_expert || at.group != held_group || panel != held_panel) {
                // the rows of x are not those that shared memory holds, or not in that order
                bool other = panel != held_panel;
                __syncthreads();
                if (at.expert != held_expert || at.group != held_group) {
                    if (threadIdx.x < 8 * NB) {
                        const int c = threadIdx.x;
                        int from = -1, to = -1;
                        if (c < cols) {
                            const int pair = p.plan.pairs[first + c];
                            if (pair >= 0 && pair < p.plan.pairs_total) {
                                from = GEGLU ? pair / p.plan.topk : first + c;
                                to = GEGLU ? first + c : pair;
                            } else {
                                record_error(p.ctx, kDevErrIndex);
                            }
                        }
                        other |= held_expert < 0 || src[c] != from;  // experts of one token have one row
                        src[c] = from;
                        dst[c] = to;
                    }
                    other = __syncthreads_or(other);
                }
                if (other)
                    for (int u = warp; u < (c1 - c0) * used; u += warps) {
                        const int n = u % used, c = u / used;
                        const int row = src[n * C::pairs + g % C::pairs];
                        // addresses count from the panel's first chunk
                        char *xp = xs - static_cast<int64_t>(c0) * 8 * L::x_block;
                        float *sp = scale - c0 * 8 * C::blocks;
                        using T = std::conditional_t<PARTS == 1, uint16_t, float>;
                        stage_x<NB>(p, xp, sp, row < 0 ? nullptr : static_cast<const T *>(p.x) + row * p.x_stride, c0 + c, n, lane);
                    }
                held_expert = at.expert;
                held_group = at.group;
                held_panel = panel;
                __syncthreads();
            }
            for (int c = c0 + (kw - c0 % p.kw + p.kw) % p.kw; c < c1; c += p.kw) {
                if (c + p.kw < p.chunks) {
                    load(at, c + p.kw, done + 1);
                } else {
                    advance<NB>(p, next);
                    load(next, kw, done + 1);
                }
                if constexpr (ALIGNED) {
                    if (there && ok) {
                        const int slot = done & (kStages - 1);
                        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&bars[warp][slot], parity >> slot & 1u, p.ctx));
                        parity ^= 1u << slot;
                    }
                } else {
                    copy_wait<1>();
                    __syncwarp();
                }
                if (there && ok) {
                    auto products = [&](auto blocks) {
                        stage_products<PARTS == 1, C::parts, C::blocks, decltype(blocks)::value, ALIGNED>(
                            ring_ptr + (done & 1) * L::stage, xs + (c - c0) * 8 * L::x_block, scale + (c - c0) * 8 * C::blocks,
                            min(8, p.blocks - c * 8), skew, p.magic, lane, total);
                    };
                    if (C::blocks > 1 && used == 1)
                        products(std::integral_constant<int, 1>());
                    else
                        products(std::integral_constant<int, C::blocks>());
                }
                __syncwarp();
                ++done;
            }
        }
        if constexpr (C::split)  // both parts of columns 2 t and 2 t + 1
#pragma unroll
            for (int n = 0; n < C::blocks; ++n)
                if (n < used)
#pragma unroll
                    for (int r = 0; r < kTiles; ++r)
#pragma unroll
                        for (int i = 0; i < 4; ++i) total[r][n][i] += __shfl_xor_sync(0xFFFFFFFFu, total[r][n][i], 2);
        // the item's sums: element (r, n, i) of lane is row 16 r + 8 (i / 2) + g, column 2 t + i % 2 of block n
        auto store = [&](int r, int n, int i, int l, float a, float b) {
            const int64_t row = row0 + 16 * r + 8 * (i >> 1) + (l >> 2);
            const int to = dst[n * C::pairs + 2 * (l & 3) + (i & 1)];
            if (to >= 0 && row < p.n) put(p.out, to * p.out_stride + row, p.out_bf16, GEGLU ? gelu(a) * b : a);
        };
        const bool own = !C::split || t < 2;  // sums that no other lane has too
        if (p.kw > 1) {
            constexpr int kTileWords = C::lanes * 4, kBlockWords = kTiles * kTileWords, kWords = C::blocks * kBlockWords;
            float *mine = part + warp * kWords;
            barrier(1 + rw, p.kw * 32);  // the last item's sums are read
#pragma unroll
            for (int n = 0; n < C::blocks; ++n)
                if (own && n < used)
#pragma unroll
                    for (int r = 0; r < kTiles; ++r)
                        reinterpret_cast<float4 *>(mine + n * kBlockWords + r * kTileWords)[C::split ? 2 * g + t : lane] =
                            make_float4(total[r][n][0], total[r][n][1], total[r][n][2], total[r][n][3]);
            barrier(1 + rw, p.kw * 32);
            const float *all = part + rw * p.kw * kWords;
            if (there)
                for (int v = kw * 32 + lane; v < used * kPairs * kTileWords; v += p.kw * 32) {
                    const int n = v / (kPairs * kTileWords), in = v % (kPairs * kTileWords);
                    const float *from = all + n * kBlockWords + in;
                    float a = 0.0f, b = 0.0f;
                    for (int w = 0; w < p.kw; ++w) {
                        a += from[w * kWords];
                        if constexpr (GEGLU) b += from[w * kWords + kPairs * kTileWords];
                    }
                    const int l = (in >> 2) % C::lanes;
                    store(in / kTileWords, n, in & 3, C::split ? (l >> 1) * 4 + (l & 1) : l, a, b);
                }
        } else if (there && own) {
#pragma unroll
            for (int n = 0; n < C::blocks; ++n)
                if (n < used)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int r = 0; r < kPairs; ++r) store(r, n, i, lane, total[r][n][i], total[GEGLU ? r + kPairs : r][n][i]);
        }
        at = next;
    }
    if constexpr (ALIGNED) {
        // a copy may still be on its way where a wait ran out; once more, with the same limit
        if (!ok && lane < kStages) wait_drain(smem_addr(&bars[warp][lane]), parity >> lane & 1u, p.ctx);
        __syncwarp();
    } else {
        copy_wait<0>();
    }
}

constexpr int kSharedLimit = 232448 - 256;  // beside the kernel's own

template <int PARTS, int NB, bool GEGLU, bool ALIGNED>
cudaError_t launch_stream(StreamParams p, cudaStream_t stream) {
    using L = StreamLayout<PARTS, NB, ALIGNED>;
    static int limits[kMaxDevices];
    // as many warps as fit beside all of x, four at least, and x in panels beyond that
    int warps = kMaxWarps;
    p.x_panel = p.chunks;
    while (warps > 4 && L::total(warps, p.x_panel) > kSharedLimit) warps -= 2;
    while (L::total(warps, p.x_panel) > kSharedLimit) --p.x_panel;
    // How many warps share an item: many where there are few items (their chunks
    // follow one another), few where there are many (their sums meet).  A block takes
    // its items in whole turns; a turn costs its chunks and about 1.2 chunks' time for
    // x and the sums.  The number of items is what pairs spread at random would give:
    // an expert is met with 1 - (1 - topk / experts)^tokens, and a count of many pairs
    // leaves its last tile half full.  Measured with 1, 2, 4 and 8 warps, fp32 GeGLU of 8
    // out of 64 experts of 1024 x 2048: 1 token 21.8, 14.2, 10.3 and 11.0 us, 4 tokens
    // 23.5, 26.8, 23.4, 25.7, 16 tokens 52.9, 43.4, 46.7, 53.3, 63 tokens 79, 71, 75, 86.
    constexpr int rows = GEGLU ? kRows / 2 : kRows;
    const double experts = static_cast<double>(p.plan.experts);
    const double met = 1.0 - std::pow(1.0 - p.plan.topk / experts, static_cast<double>(p.plan.pairs_total / p.plan.topk));
    const double tiles = p.plan.pairs_total / (experts * 8 * NB);
    const double units = experts * (tiles < 0.5 ? met : std::max(met, tiles + 0.5 * (1.0 - 1.0 / (8 * NB))));
    int best = 1;
    double least = 0.0;
    for (int kw = 1; kw <= std::min(p.chunks, warps); kw *= 2) {
        const int rw = warps / kw;
        const double turns = std::max(1.0, std::ceil(units * ((p.n + rows * rw - 1) / (rows * rw)) / device_sm_count()));
        const double cost = turns * ((p.chunks + kw - 1) / kw + 1.2);
        if (kw == 1 || cost < least) {
            best = kw;
            least = cost;
        }
    }
    p.kw = best;
    p.rw = warps / p.kw;
    p.row_groups = static_cast<int>((p.n + rows * p.rw - 1) / (rows * p.rw));
    warps = p.rw * p.kw;
    const int smem = L::total(warps, p.x_panel);
    const cudaError_t e = ensure_smem(stream_kernel<PARTS, NB, GEGLU, ALIGNED>, smem, false, limits);
    if (e != cudaSuccess) return e;
    CUtensorMap w0 = {}, w1 = {};
    if constexpr (ALIGNED) {
        const uint64_t all = static_cast<uint64_t>(p.plan.experts) * p.n;
        if (!encode_tmap_2d(&w0, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.w[0], p.row_bytes, all, p.row_bytes, 144, rows) ||
            !encode_tmap_2d(&w1, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.w[GEGLU ? 1 : 0], p.row_bytes, all, p.row_bytes, 144, rows))
            return cudaErrorInvalidValue;
    }
    return launch_kernel(stream_kernel<PARTS, NB, GEGLU, ALIGNED>, dim3(device_sm_count()), dim3(warps * 32), smem, stream,
                         1, w0, w1, p);
}

template <bool GEGLU, bool ALIGNED, int NB>
cudaError_t launch_parts(const StreamParams &p, cudaStream_t stream) {
    return p.x_bf16 ? launch_stream<1, NB, GEGLU, ALIGNED>(p, stream) : launch_stream<2, NB, GEGLU, ALIGNED>(p, stream);
}

// Groups of 16 pairs where the experts have more than eight on average.
template <bool GEGLU>
cudaError_t launch_form(StreamParams &p, cudaStream_t stream) {
    p.blocks = static_cast<int>(p.k / kQK);
    p.chunks = (p.blocks + 7) / 8;
    p.row_bytes = static_cast<int64_t>(p.blocks) * kQ4_0Bytes;
    p.matrix_bytes = p.row_bytes * p.n;
    p.w_bytes = p.matrix_bytes * p.plan.experts;
    p.magic = p.x_bf16 ? 0x41804180u : 0x64006400u;
    p.x_wide = reinterpret_cast<uintptr_t>(p.x) % (p.x_bf16 ? 8 : 16) == 0 && p.x_stride % 4 == 0;  // loads of four
    const bool aligned = p.k % kChunk == 0 && p.plan.experts * p.n < (int64_t(1) << 31);  // a box's row is 32 bits
    const bool many = p.plan.pairs_total > 8 * static_cast<int64_t>(p.plan.experts);
    if (aligned) return many ? launch_parts<GEGLU, true, 2>(p, stream) : launch_parts<GEGLU, true, 1>(p, stream);
    return many ? launch_parts<GEGLU, false, 2>(p, stream) : launch_parts<GEGLU, false, 1>(p, stream);
}

}  // namespace experts
}  // namespace qmm
