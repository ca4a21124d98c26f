// qmm_attn.cu -- attention over the paged Q4_0 cache (include/qmm.h,
// qmm_attn_q4_0): the streaming form, for single tokens and small groups of
// query rows.
//
// Mathematics.  With codes n (0..15) and scales d of 32-value blocks b,
//   s_j = scale * sum_b d_jb * sum_i (n_jbi - 8) q_bi
//   o_i = sum_j (p_j d_jb) (n_jbi - 8),  p_j = 2^(s_j log2(e) - M)
// so both products have small integers on the cache's side and the scales
// leave them: K's multiply fp32 block sums, V's join the softmax weights.
// The integers are exact in binary16, therefore the products run on
// mma.sync m16n8k16 with the cache as the 16-row operand, taken from the
// 4-bit codes in registers.  For bf16 outputs a code masked in place is a
// subnormal binary16 number (n * 2^-24, or 16 n * 2^-24 for the upper of two),
// the powers of two being folded into q or undone at the end; fp32 outputs
// take two more instructions for normal numbers, because the tensor cores'
// sums of subnormal operands keep some 18 bits (6e-6 of the output, measured).
// tcgen05 would need those
// operands written out to shared or tensor memory first, 3.6 times the bytes
// of the codes, for 8 columns that it cannot fill.
//
// Precision.  fp32 output: q and p*d enter as two binary16 parts each (22
// bits) in neighbouring columns, four query rows to 8 columns.  bf16
// output: one part (11 bits), eight rows.  Both are scaled by powers of two
// so that the largest lies below 2^15 (q per row, p*d per tile and block of 32
// values).  Weights below 2^-24 of a tile's largest, which binary16 would lose, take a second
// pass over the tile's values.  V's sums run over 64 keys in the tensor
// core, then join the fp32 running output.
//
// Work.  The keys of all (request, key head, row group) items, in tiles of
// 64 keys, form one line that is cut into equal parts for all warps of a
// grid that fills the GPU, whatever the lengths are.  Each warp streams its
// tiles through its own shared-memory buffers (16-byte asynchronous copies,
// placed so that ldmatrix reads them without conflicts): while it works on a
// tile's values the next tile's keys arrive, and the other way round.  TMA
// boxes of the 32 to 128 byte rows kept the warps waiting to issue them, 4700
// of 13000 cycles a tile.  An item that several warps share leaves
// a maximum, a sum and an unnormalised output per warp; a CTA joins what its
// warps hold, and a second kernel joins what several CTAs hold.
//
// Bound, at head_dim 128 in bf16, by the instructions that turn codes into
// operands and by their dependencies (56 % of the issue slots, 48 % of DRAM's
// rate); at head_dim 256 in fp32 by latency: two warps an SM quarter issue in
// 33 % of the slots and wait longest for instructions to be fetched.
// Measured, both kernels: 128 requests of up to 8192 keys, 16 heads on 4 of
// 128, bf16, 91.5 us (329 MB, 3.6 TB/s); fp32 outputs, 8 heads on 2 of 256: one
// request of 131071 keys 40.7 us (75 MB), 16 of up to 4097 17.7 us, one of 301
// 13 us.  Scores that spread by more than 23 powers of two within a tile take
// further passes over its values: by their standard deviation 1.2, 2.4, 4 and
// 8 the 128 requests (from a flushed L2) 101, 112, 138 and 178 us, the 131071
// keys 59, 62, 68 and 87.
#include "qmm_attn.cuh"

#include <algorithm>

namespace qmm {
namespace {

constexpr int kWarps = 8;  // of a CTA, at most
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 64;  // keys
constexpr float kFaint = 1.0f / 16777216.0f;  // 2^-24
constexpr uint32_t kMinus8 = 0x80088008u, kMinus128 = 0x80808080u;  // binary16 pairs, times 2^-24

// One head dimension's shared memory, per warp.
template <int D, int NT, bool EXACT>
struct Layout {
    static constexpr int NB = D / 32;
    static constexpr int rows = EXACT ? 4 * NT : 8 * NT;  // query rows of an item
    static constexpr int codes = kTile * D / 2, scales = kTile * NB * 2;
    static constexpr int p_stride = kTile + 8;  // floats
    // the code buffers lie in front of everything, 1024-byte aligned; together
    // they have room for a partial record
    static constexpr int code_bytes = 2 * codes;
    // the rest, from its own start
    static constexpr int v_scales = scales;
    static constexpr int q = v_scales + scales;          // B fragments [NT][NB][32 lanes] x 16 bytes
    static constexpr int bias = q + NT * NB * 512;       // -8 sum q [NT][NB][4 lanes] x {c0, c1, c0, c1}, bf16 only
    static constexpr int d = bias + (EXACT ? 0 : NT * NB * 64);        // V's scales by block: pairs of keys, binary16 or fp32
    static constexpr int p = d + NB * kTile * (EXACT ? 4 : 2);  // weights [rows][p_stride], EXACT only
    static constexpr int unit = p + (EXACT ? rows * p_stride * 4 : 0);  // of V's blocks, fp32
    static constexpr int rest_bytes = unit + (NB * 4 + 15) / 16 * 16;
    // CTAs on an SM: as the registers of the accumulators allow
    static constexpr int ctas = D == 256 ? 1 : D == 128 && NT == 2 ? 1 : 2;
    static constexpr int fit = (232448 / ctas - 1024 - 14336) / (code_bytes + rest_bytes);
    static constexpr int warps = fit < kWarps ? fit : kWarps;  // as many as fit shared memory
    static constexpr int threads = warps * 32;
    static_assert(rows * D * 4 <= code_bytes, "a partial record fits the code buffers");
    static_assert(rest_bytes % 16 == 0, "alignment of the next warp's part");
};

// Where an item's rows go.
struct Target {
    int row0, rows, kv_head, group;
};

// A warp holds at most two parts of items that it shares with others: one
// that an earlier warp began (head), and one that a later warp goes on with
// (tail; always its last).
enum : int {
    kHead = 1,        // there is a head part
    kHeadOpen = 2,    // ... which a later warp goes on with
    kHeadLast = 4,    // ... and which is the warp's last part
    kTail = 8,        // there is a tail part
    kEmpty = 16       // no tiles at all
};

// One request as the line sees it.
struct Request : RequestRows {
    int tile0, tiles;    // of every item of the request
    int groups;          // row groups
};

// A warp's place in the line and the part that it works on.
struct Part {
    int64_t x, end;
    int t0, t1, tiles;  // tiles of the item
    Target to;
    int b;                       // request
    int lo, hi, lo_all, hi_all;  // keys that any, and that every, row sees
    int row_lo[8], row_hi[8];    // keys that each row sees
};

// What the CTA's threads share, after the warps' buffers.
struct Shared {
    int64_t prefix[kThreads];   // line places before each thread's requests
    Request request[kThreads];  // the requests, where every thread has at most one
    int64_t scratch[kWarps][2];
    int flags[kWarps];
    Part part[kWarps];             // what a warp is at, kept out of its registers
    Target target[kWarps][2];      // of head and tail
    float stat[kWarps][2][8][2];   // maximum and sum of each row
    float weight[8][kWarps];       // of a chain's parts, by row
    float total[8][2];             // its maximum and sum
};

// A CTA's parts in global memory, the same way: flags and the tail's target.
struct CtaParts {
    int flags;
    Target target;
};

struct StreamParams {
    AttnArgs a;
    const uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
    int num_pages, page_shift, kv_heads;
    bool q_pairs;         // rows of q are aligned to two values
    uint32_t magic;       // 1024, 1024 in binary16: a register where a constant would cost an instruction
    float *warp_records;  // [CTAs * kWarps]: head parts that are not the last
    float *cta_records;   // [CTAs][2]: head and tail part
    CtaParts *parts;      // [CTAs]
    LaunchCtx ctx;
};

// Floats of one record in global memory: outputs [rows][D] and then maximum
// and sum [rows][2], at most 8 rows of 256.
constexpr int kRecord = 8 * 256 + 16;
constexpr int kRecordStat = 8 * 256;

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
// d = a b + c: 16 x 16 by 16 x 8, binary16 with fp32 sums
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1, float c0, float c1, float c2, float c3) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
// the transpose of an 8 x 8 matrix of binary16, a row's pair per lane
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
// 0xFFFF in each half that is not zero (NaN is not)
__device__ __forceinline__ uint32_t not_zero2(uint32_t v) {
    return __hneu2_mask(*reinterpret_cast<const __half2 *>(&v), __half2half2(__ushort_as_half(0)));
}

// ---- the line of tiles -----------------------------------------------------------

// The number of tiles up to key n.
__device__ __forceinline__ int tiles_to(int n) { return (n + kTile - 1) / kTile; }

template <int ROWS>
__device__ __forceinline__ Request request(const StreamParams &p, int b) {
    const AttnArgs &a = p.a;
    Request r;
    static_cast<RequestRows &>(r) = request_rows(a, p.page_shift, b);
    r.tile0 = first_key(a, r.first) / kTile;
    r.tiles = max(1, tiles_to(r.len) - r.tile0);
    r.groups = (r.rows * (a.heads / p.kv_heads) + ROWS - 1) / ROWS;
    return r;
}

// The line: where each warp's tiles lie.  Places are tiles; in the spread
// form an item takes a whole number of CTAs' warps, one tile each.
struct Line {
    int64_t total;
    bool spread;
};

// Places of one item.
template <int W>
__device__ __forceinline__ int item_places(const Request &r, bool spread) {
    return spread ? (r.tiles + W - 1) / W * W : r.tiles;
}

// Fills sh.prefix (and sh.request).  Spread is taken when no warp then gets
// more than one tile: an item of few tiles is then joined within its CTA.
template <int ROWS, int W>
__device__ __forceinline__ Line build_line(const StreamParams &p, Shared &sh) {
    constexpr int threads = W * 32;
    const int per = (p.a.batch + threads - 1) / threads;
    const int b0 = min(p.a.batch, static_cast<int>(threadIdx.x) * per), b1 = min(p.a.batch, b0 + per);
    int64_t tiles = 0, places = 0;
    int bad = 0;
    for (int b = b0; b < b1; ++b) {
        const Request r = request<ROWS>(p, b);
        const int64_t items = static_cast<int64_t>(r.groups) * p.kv_heads;
        tiles += items * r.tiles;
        places += items * item_places<W>(r, true);
        bad |= r.bad;
        if (per == 1) sh.request[threadIdx.x] = r;
    }
    if (bad && blockIdx.x == 0) record_error(p.ctx, kDevErrIndex);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t sum[2] = {tiles, places};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xFFFFFFFFu, sum[0], o), y = __shfl_up_sync(0xFFFFFFFFu, sum[1], o);
        if (lane >= o) {
            sum[0] += x;
            sum[1] += y;
        }
    }
    if (lane == 31) {
        sh.scratch[warp][0] = sum[0];
        sh.scratch[warp][1] = sum[1];
    }
    __syncthreads();
    int64_t before[2] = {0, 0}, total[2] = {0, 0};
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (w < warp) before[i] += sh.scratch[w][i];
            total[i] += sh.scratch[w][i];
        }
    const bool spread = total[1] <= static_cast<int64_t>(gridDim.x) * W;
    sh.prefix[threadIdx.x] = spread ? before[1] + sum[1] - places : before[0] + sum[0] - tiles;
    __syncthreads();
    return Line{spread ? total[1] : total[0], spread};
}

// The request that holds place x of the line, and the places before it.
template <int ROWS, int W>
__device__ __forceinline__ int find_request(const StreamParams &p, const Shared &sh, const Line &line, int64_t x,
                                            int64_t &before, Request &r) {
    constexpr int threads = W * 32;
    // the last thread whose prefix is at most x holds it: 8 ranges a lane
    const int lane = threadIdx.x & 31;
    int count = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) count += __popc(__ballot_sync(0xFFFFFFFFu, sh.prefix[i * 32 + lane] <= x));
    const int at = count - 1, per = (p.a.batch + threads - 1) / threads;
    before = sh.prefix[at];
    if (per == 1) {
        r = sh.request[at];
        return at;
    }
    for (int b = at * per;; ++b) {
        r = request<ROWS>(p, b);
        const int64_t n = static_cast<int64_t>(item_places<W>(r, line.spread)) * r.groups * p.kv_heads;
        if (x < before + n || b + 1 >= p.a.batch) return b;
        before += n;
    }
}

// An item: a key head and a group of rows of one request.
struct Item {
    int b, kv_head, group;
};

// ---- one warp's tiles -------------------------------------------------------------

template <int D, int NT, bool EXACT>
struct WarpState {
    using L = Layout<D, NT, EXACT>;
    static constexpr int NB = L::NB;
    static constexpr int R = EXACT ? 1 : 2;  // query rows per lane and column tile

    uint8_t *codes, *rest;
    int lane, g, t;
    // running statistics of this lane's rows: maximum and sum of the weights
    // 2^(s - top)
    float top[NT][R], sum[NT][R];
    float2 out[NT][NB][2][2];         // [block][even, odd value][value i, 16 + i (x 16)]: two columns
    float unit[NT][R];                // score = sum * unit > 0
};

// Page indices of the keys ahead: lane i holds page first + i of the request.
struct Pages {
    int32_t lane_page;
    int first;
};

__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t *src) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the latest group of this thread's copies are there, for the warp.
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncwarp();
}

// By how much the 16-byte chunks of a row of codes are rotated (exclusive or),
// so that eight rows' chunks of one block lie in different banks.
template <int D>
__device__ __forceinline__ int chunk_swizzle(int row) {
    return D == 256 ? (row & 7) : D == 128 ? ((row >> 1) & 3) : ((row >> 2) & 1);
}

// Starts the copies of the codes and scales of tile [key0, key0 + 64), those
// of 16-key groups that hold keys of [lo, hi) and have a page, as one group.
template <int D>
__device__ __forceinline__ void fetch_tile(const StreamParams &p, const uint8_t *codes, const uint8_t *scales,
                                           uint32_t codes_to, uint32_t scales_to, int kv_head, int key0, int lo, int hi,
                                           const Pages &pages, int lane) {
    constexpr int row_bytes = D / 2, group_bytes = 16 * row_bytes, scale_bytes = D / 16;  // of a row, 16 rows, a row
    const int shift = p.page_shift, mask = (1 << shift) - 1;
    if (shift >= 6) {  // the tile lies in one page
        const int32_t page = __shfl_sync(0xFFFFFFFFu, pages.lane_page, (key0 >> shift) - pages.first);
        if (page >= 0 && page < p.num_pages) {
            const int64_t row = ((page * p.kv_heads + kv_head) << shift) + (key0 & mask);
            const uint8_t *src = codes + row * row_bytes + lane * 16;
            const int r0 = lane / (row_bytes / 16), c = lane % (row_bytes / 16);
#pragma unroll
            for (int j = 0; j < 4 * group_bytes / 512; ++j) {
                const int r = r0 + j * (512 / row_bytes);
                copy16(codes_to + r * row_bytes + ((c ^ chunk_swizzle<D>(r)) << 4), src + j * 512);
            }
            const uint8_t *from = scales + row * scale_bytes + lane * 16;
#pragma unroll
            for (int j = 0; j < (D + 127) / 128; ++j)
                if (D >= 128 || lane < D / 4) copy16(scales_to + (lane + 32 * j) * 16, from + j * 512);
        }
        copies_commit();
        return;
    }
    // lane i < 4: the row of the cache where group i begins, or -1
    const int key = key0 + 16 * (lane & 3);
    const int32_t page = __shfl_sync(0xFFFFFFFFu, pages.lane_page, ((key >> shift) - pages.first) & 31);
    int row = -1;
    if (key < hi && key + 16 > lo && page >= 0 && page < p.num_pages)
        row = (((page * p.kv_heads) + kv_head) << shift) + (key & mask);  // below 2^31
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const int at = __shfl_sync(0xFFFFFFFFu, row, g);
        if (at < 0) continue;
        const uint8_t *src = codes + static_cast<int64_t>(at) * row_bytes + lane * 16;
#pragma unroll
        for (int j = 0; j < group_bytes / 512; ++j) {
            const int r = (lane + 32 * j) / (row_bytes / 16), c = (lane + 32 * j) % (row_bytes / 16);
            copy16(codes_to + (16 * g + r) * row_bytes + ((c ^ chunk_swizzle<D>(r)) << 4), src + j * 512);
        }
    }
    // the scales: chunk i of the tile's 4 D bytes, in group i / (D / 16)
#pragma unroll
    for (int j = 0; j < (D + 127) / 128; ++j) {
        const int i = lane + 32 * j, g = i / (D / 16);
        const int at = __shfl_sync(0xFFFFFFFFu, row, g & 3);
        if (at >= 0 && i < D / 4)
            copy16(scales_to + i * 16, scales + static_cast<int64_t>(at) * scale_bytes + (i % (D / 16)) * 16);
    }
    copies_commit();
}

// The lane's D / 32 consecutive values of each of the item's rows of q: they
// lie in one block.
template <int D, int NT, bool EXACT>
struct QueryRows {
    float v[Layout<D, NT, EXACT>::rows][D / 32];
    int pos[Layout<D, NT, EXACT>::rows];
};

template <int D, int NT, bool EXACT>
__device__ __forceinline__ void load_q(const StreamParams &p, QueryRows<D, NT, EXACT> &q, const Request &r,
                                       const Item &it, int lane) {
    constexpr int ROWS = Layout<D, NT, EXACT>::rows, E = D / 32;
    const AttnArgs &a = p.a;
    const int heads = a.heads / p.kv_heads, all = r.rows * heads;
#pragma unroll
    for (int row = 0; row < ROWS; ++row) {
        const int flat = min(it.group * ROWS + row, all - 1), token = flat / heads;  // past the end: the last again
        const int64_t at = (static_cast<int64_t>(r.row0) + token) * a.q_stride +
                           static_cast<int64_t>(it.kv_head * heads + flat - token * heads) * D + lane * E;
        q.pos[row] = r.first + token;
        if (p.q_pairs) {  // rows are aligned to pairs of values
#pragma unroll
            for (int i = 0; i < E; i += 2) {
                if (a.q_bf16) {
                    const uint32_t u = *reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(a.q) + at + i);
                    q.v[row][i] = __uint_as_float(u << 16);
                    q.v[row][i + 1] = __uint_as_float(u & 0xFFFF0000u);
                } else {
                    const float2 u = *reinterpret_cast<const float2 *>(static_cast<const float *>(a.q) + at + i);
                    q.v[row][i] = u.x;
                    q.v[row][i + 1] = u.y;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) q.v[row][i] = load_value(a.q, at + i, a.q_bf16);
        }
    }
}

template <int D, int NT, bool EXACT>
__device__ __forceinline__ void stage_zero(WarpState<D, NT, EXACT> &w, Part &part, int row) {
    using L = Layout<D, NT, EXACT>;
    constexpr int NB = L::NB;
    const int nt = row / (L::rows / NT), in = row % (L::rows / NT), cols = EXACT ? 2 : 1;
    uint4 *frag = reinterpret_cast<uint4 *>(w.rest + L::q) + nt * NB * 32 + in * cols * 4;
    for (int i = w.lane; i < NB * cols * 4; i += 32)
        frag[i / (cols * 4) * 32 + i % (cols * 4)] = make_uint4(0u, 0u, 0u, 0u);
    if constexpr (!EXACT) {
        float *bias = reinterpret_cast<float *>(w.rest + L::bias) + nt * NB * 16 + (in >> 1) * 4 + (in & 1);
        for (int i = w.lane; i < NB; i += 32) bias[i * 16] = bias[i * 16 + 2] = 0.0f;
    }
    if (w.lane == 0) {
        part.row_lo[row] = part.row_lo[0];
        part.row_hi[row] = part.row_hi[0];
    }
}

// Those rows as B fragments, scaled to below 2^15, with -8 times the block
// sums (the codes are used as 0..15).
template <int D, int NT, bool EXACT>
__device__ __forceinline__ void stage_q(const StreamParams &p, WarpState<D, NT, EXACT> &w,
                                        QueryRows<D, NT, EXACT> &rows, Part &part, const Request &r, int rows_here) {
    using L = Layout<D, NT, EXACT>;
    constexpr int NB = L::NB, E = D / 32;
    const AttnArgs &a = p.a;
    float (&v)[L::rows][E] = rows.v;
    const int (&pos)[L::rows] = rows.pos;
    uint32_t *frag = reinterpret_cast<uint32_t *>(w.rest + L::q);
    float *bias = reinterpret_cast<float *>(w.rest + L::bias);
    const int d0 = w.lane * E, block = d0 / 32;
    // the sign of the scale goes to q; a scale of 0 takes q with it
    const float size = fabsf(a.scale) * kLog2e, sign = a.scale < 0.0f ? -1.0f : a.scale == 0.0f ? 0.0f : 1.0f;
#pragma unroll
    for (int row = 0; row < L::rows; ++row) {
        if (row >= rows_here) {  // columns without a row: zeros, which see what row 0 sees
            stage_zero<D, NT, EXACT>(w, part, row);
            continue;
        }
        uint32_t bits = 0;  // of the largest value: positive numbers order as their bits do
#pragma unroll
        for (int i = 0; i < E; ++i) {
            v[row][i] *= sign;
            bits = max(bits, __float_as_uint(v[row][i]) & 0x7FFFFFFFu);
        }
        const float big = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, bits));
        const int up = query_raise(big, size);
        const float f = pow2i(up), unit = score_unit(size, (EXACT ? 0 : 24) - up);
        const int nt = row / (L::rows / NT), in = row % (L::rows / NT);
        float s_hi = 0.0f;
        // value d of a block: lane (d & 15) / 4 of the column, register
        // (d & 1) * 2 + d / 16, half (d / 2) & 1; a lane's values share d / 16
        const int high = (d0 >> 4) & 1;
        const float f16 = f * (!EXACT && high ? 0.0625f : 1.0f), back = high ? 16.0f : 1.0f;
        float one[E], two[E];
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float x = v[row][i] * f16;
            one[i] = __half2float(EXACT ? __float2half_rz(x) : __float2half_rn(x));
            two[i] = EXACT ? __half2float(__float2half_rn(x - one[i])) : 0.0f;
            s_hi += one[i] * back;
        }
        uint32_t *to = frag + ((nt * NB + block) * 32 + (EXACT ? in * 2 : in) * 4) * 4;
        if constexpr (E >= 4) {
#pragma unroll
            for (int i = 0; i < E; i += 4) {
                uint32_t *at = to + (((d0 + i) & 15) >> 2) * 4 + high;
                at[0] = pack_rn(one[i], one[i + 2]);
                at[2] = pack_rn(one[i + 1], one[i + 3]);
                if constexpr (EXACT) {  // the next column: four lanes of four registers further
                    at[16] = pack_rn(two[i], two[i + 2]);
                    at[18] = pack_rn(two[i + 1], two[i + 3]);
                }
            }
        } else {  // two values: 0 1 or 2 3 of a quad
            __half *at = reinterpret_cast<__half *>(to + ((d0 & 15) >> 2) * 4 + high) + ((d0 >> 1) & 1);
            at[0] = __float2half_rn(one[0]);
            at[4] = __float2half_rn(one[1]);
            if constexpr (EXACT) {
                at[32] = __float2half_rn(two[0]);
                at[36] = __float2half_rn(two[1]);
            }
        }
        if constexpr (!EXACT) {
#pragma unroll
            for (int o = 1; o < 32 / E; o <<= 1) s_hi += __shfl_xor_sync(0xFFFFFFFFu, s_hi, o);
        }
        if (!EXACT && w.lane % (32 / E) == 0) {
            const float m8 = -8.0f / 16777216.0f;
            float *b8 = bias + (nt * NB + block) * 16 + (in >> 1) * 4 + (in & 1);
            b8[0] = b8[2] = s_hi * m8;
        }
        if (w.lane == 0) {
            part.row_lo[row] = first_key(a, pos[row]);
            part.row_hi[row] = a.causal ? min(r.len, pos[row] + 1) : r.len;
        }
        // the lanes that hold this row's scores keep their unit
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < w.R; ++k)
                if (n == nt && (EXACT ? w.t : w.t * 2 + k) == in) w.unit[n][k] = unit;
    }
    __syncwarp();
}

// n - 8 of the lower and of the upper codes of a word as binary16 pairs.
// fp32 output: normal numbers, by way of 1024 + n.  A subnormal operand is
// summed with the exponent of the smallest normal number, and loses the ten
// bits between from the fp32 sums' low end.
__device__ __forceinline__ uint32_t lower8(uint32_t x, uint32_t magic) {
    return hadd2((x & 0x000F000Fu) | magic, 0xE408E408u);  // - 1032
}
__device__ __forceinline__ uint32_t upper8(uint32_t x, uint32_t magic) {
    return hfma2((x & 0x00F000F0u) | magic, 0x2C002C00u, 0xD480D480u);  // / 16 - 72
}

// NB binary16 scales of one key.
template <int NB>
__device__ __forceinline__ void load_scales(const uint16_t *row, uint32_t (&d)[NB / 2]) {
    if constexpr (NB == 8) {
        const uint4 v = *reinterpret_cast<const uint4 *>(row);
        d[0] = v.x; d[1] = v.y; d[2] = v.z; d[3] = v.w;
    } else if constexpr (NB == 4) {
        const uint2 v = *reinterpret_cast<const uint2 *>(row);
        d[0] = v.x; d[1] = v.y;
    } else {
        d[0] = *reinterpret_cast<const uint32_t *>(row);
    }
}

// Sums of the tile before their unit: s[nt][mt][row of pair][key g, g + 8].
template <int D, int NT, bool EXACT>
__device__ __forceinline__ void tile_scores(WarpState<D, NT, EXACT> &w, uint32_t magic,
                                            float (&s)[NT][4][WarpState<D, NT, EXACT>::R][2]) {
    using L = Layout<D, NT, EXACT>;
    constexpr int NB = L::NB;
    const uint4 *frag = reinterpret_cast<const uint4 *>(w.rest + L::q) + w.lane;
    const float4 *bias = reinterpret_cast<const float4 *>(w.rest + L::bias) + w.t;
    const uint16_t *ks = reinterpret_cast<const uint16_t *>(w.rest);
    const int sw = chunk_swizzle<D>(w.lane);
    const uint32_t base = smem_addr(w.codes) + w.lane * (D / 2);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        // scales of keys 32 half + {0, 8, 16, 24} + g
        uint32_t d[4][NB / 2];
#pragma unroll
        for (int k = 0; k < 4; ++k) load_scales<NB>(ks + (half * 32 + k * 8 + w.g) * NB, d[k]);
        float acc[NT][2][4];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            uint32_t c[4];
            ldsm4(c, base + half * 32 * (D / 2) + ((b ^ sw) << 4));
            uint4 q[NT];
            float4 c8[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                q[n] = frag[(n * NB + b) * 32];
                if constexpr (!EXACT) c8[n] = bias[(n * NB + b) * 4];
            }
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const uint32_t x = c[2 * m], y = c[2 * m + 1], x8 = x >> 8, y8 = y >> 8;
                uint32_t k1[4], k2[4];  // A operands: the values of the first and of the second product
                if constexpr (EXACT) {
                    k1[0] = lower8(x, magic), k1[1] = lower8(y, magic), k1[2] = upper8(x, magic), k1[3] = upper8(y, magic);
                    k2[0] = lower8(x8, magic), k2[1] = lower8(y8, magic), k2[2] = upper8(x8, magic), k2[3] = upper8(y8, magic);
                } else {
                    k1[0] = x & 0x000F000Fu, k1[1] = y & 0x000F000Fu, k1[2] = x & 0x00F000F0u, k1[3] = y & 0x00F000F0u;
                    k2[0] = x8 & 0x000F000Fu, k2[1] = y8 & 0x000F000Fu, k2[2] = x8 & 0x00F000F0u, k2[3] = y8 & 0x00F000F0u;
                }
                const uint32_t dx = d[2 * m][b / 2], dy = d[2 * m + 1][b / 2];
                const float df = b & 1 ? high_float(dx) : low_float(dx), dg = b & 1 ? high_float(dy) : low_float(dy);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float z[4];
                    if constexpr (EXACT)
                        mma16816(z, k1[0], k1[1], k1[2], k1[3], q[n].x, q[n].y, 0.0f, 0.0f, 0.0f, 0.0f);
                    else
                        mma16816(z, k1[0], k1[1], k1[2], k1[3], q[n].x, q[n].y, c8[n].x, c8[n].y, c8[n].z, c8[n].w);
                    mma16816(z, k2[0], k2[1], k2[2], k2[3], q[n].z, q[n].w, z[0], z[1], z[2], z[3]);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[n][m][i] = b ? fmaf(i < 2 ? df : dg, z[i], acc[n][m][i]) : (i < 2 ? df : dg) * z[i];
                }
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if constexpr (EXACT) {
                        s[n][half * 2 + m][0][h] = acc[n][m][2 * h] + acc[n][m][2 * h + 1];
                    } else {
                        s[n][half * 2 + m][0][h] = acc[n][m][2 * h];
                        s[n][half * 2 + m][1][h] = acc[n][m][2 * h + 1];
                    }
                }
    }
}

// V's scales, by block and in the order the B operand takes keys: 0 1 8 9
// 2 3 10 11 ... of each 16.  They are scaled so that the block's largest lies
// in [1, 2) (binary16) or [2^14, 2^15) (fp32), and 0 where `seen` has no bit
// for the key (bit i: key 2 lane + i).  Each block has a unit of its own: one
// for all would take the low bits of p d from the outputs of small blocks.
template <int D, int NT, bool EXACT>
__device__ __forceinline__ void tile_scales(WarpState<D, NT, EXACT> &w, unsigned seen) {
    using L = Layout<D, NT, EXACT>;
    constexpr int NB = L::NB;
    const uint16_t *vs = reinterpret_cast<const uint16_t *>(w.rest + L::v_scales) + w.lane * 2 * NB;
    uint32_t d[2][NB / 2];
    load_scales<NB>(vs, d[0]);
    load_scales<NB>(vs + NB, d[1]);
    int e[NB];  // exponents of the blocks' largest
#pragma unroll
    for (int i = 0; i < NB / 2; ++i) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (!((seen >> k) & 1u)) d[k][i] = 0u;
        // NaN is passed over, and infinity counts as 65504; the order of positive
        // numbers is that of their bits
        const uint32_t big = hmin2(hmax2(hmax2(d[0][i] & 0x7FFF7FFFu, d[1][i] & 0x7FFF7FFFu), 0u), 0x7BFF7BFFu);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, h ? big >> 16 : big & 0xFFFFu);
            e[2 * i + h] = top ? exponent(low_float(top)) : 0;
        }
    }
    float *unit = reinterpret_cast<float *>(w.rest + L::unit);
#pragma unroll
    for (int b = 0; b < NB; ++b)
        if (w.lane == b) unit[b] = pow2i(e[b]);
    const int i8 = w.lane >> 3, i4 = (w.lane >> 2) & 1, i2 = w.lane & 3;
    if constexpr (EXACT) {
        float2 *to = reinterpret_cast<float2 *>(w.rest + L::d) + i8 * 8 + i2 * 2 + i4;
#pragma unroll
        for (int i = 0; i < NB / 2; ++i) {
            const float up0 = pow2i(14 - e[2 * i]), up1 = pow2i(14 - e[2 * i + 1]);
            to[(2 * i) * (kTile / 2)] = make_float2(low_float(d[0][i]) * up0, low_float(d[1][i]) * up0);
            to[(2 * i + 1) * (kTile / 2)] = make_float2(high_float(d[0][i]) * up1, high_float(d[1][i]) * up1);
        }
    } else {
        uint32_t *to = reinterpret_cast<uint32_t *>(w.rest + L::d) + i8 * 8 + i2 * 2 + i4;
#pragma unroll
        for (int i = 0; i < NB / 2; ++i) {
            const float up0 = pow2i(-e[2 * i]), up1 = pow2i(-e[2 * i + 1]);
            to[(2 * i) * (kTile / 2)] = pack_rn(low_float(d[0][i]) * up0, low_float(d[1][i]) * up0);
            to[(2 * i + 1) * (kTile / 2)] = pack_rn(high_float(d[0][i]) * up1, high_float(d[1][i]) * up1);
        }
    }
}

// -(x & keep)
__device__ __forceinline__ float minus_part(float x, uint32_t keep) {
    return __uint_as_float((__float_as_uint(x) & keep) ^ 0x80000000u);
}

// out = out * f + g * unit * sum over the tile's keys of (p d) (n - 8), with the
// weights in shared memory (EXACT) or in pw, as binary16 B operands.
// EDGE: some row does not see some key of the tile, whose scale may then be
// anything.
template <int D, int NT, bool EXACT, bool EDGE>
__device__ __forceinline__ void tile_values(WarpState<D, NT, EXACT> &w, uint32_t magic, const uint32_t (&pw)[NT][4][2],
                                            const float (&f)[NT][WarpState<D, NT, EXACT>::R],
                                            const float (&g)[NT][WarpState<D, NT, EXACT>::R]) {
    using L = Layout<D, NT, EXACT>;
    constexpr int NB = L::NB;
    const float *p = reinterpret_cast<const float *>(w.rest + L::p);
    const int token = w.lane & 15, upper = w.lane >> 4;
    const int sw = chunk_swizzle<D>(token);
    const uint32_t base = smem_addr(w.codes) + L::codes + token * (D / 2);
    const uint32_t keep = EXACT && (w.g & 1) ? 0xFFFFE000u : 0u;  // odd columns hold the second part
    const float2 *unit = reinterpret_cast<const float2 *>(w.rest + L::unit);
#pragma unroll
    for (int bp = 0; bp < NB / 2; ++bp) {
        float acc[NT][2][2][4];
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            uint32_t c[4];
            ldsm4_t(c, base + ks * 16 * (D / 2) + (((2 * bp + upper) ^ sw) << 4));
            float4 pe[NT];
            if constexpr (EXACT) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    pe[n] = *reinterpret_cast<const float4 *>(p + (n * 4 + (w.g >> 1)) * L::p_stride + ks * 16 + 4 * w.t);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t x = c[2 * h], y = c[2 * h + 1], x8 = x >> 8, y8 = y >> 8;
                // bf16 output: n - 8 (lower codes) and 16 (n - 8) (upper codes), times
                // 2^-24.  -8 times the sum of the weights as a product of its own
                // would take fewer instructions, but a heavy key's code 8 must
                // leave exactly nothing.
                uint32_t xa, ya, xb, yb, xc, yc, xd, yd;
                if constexpr (EXACT) {
                    xa = lower8(x, magic), ya = lower8(y, magic), xc = lower8(x8, magic), yc = lower8(y8, magic);
                    xb = upper8(x, magic), yb = upper8(y, magic), xd = upper8(x8, magic), yd = upper8(y8, magic);
                } else {
                    xa = hadd2(x & 0x000F000Fu, kMinus8), ya = hadd2(y & 0x000F000Fu, kMinus8);
                    xb = hadd2(x & 0x00F000F0u, kMinus128), yb = hadd2(y & 0x00F000F0u, kMinus128);
                    xc = hadd2(x8 & 0x000F000Fu, kMinus8), yc = hadd2(y8 & 0x000F000Fu, kMinus8);
                    xd = hadd2(x8 & 0x00F000F0u, kMinus128), yd = hadd2(y8 & 0x00F000F0u, kMinus128);
                }
                uint32_t b0[NT], b1[NT];
                if constexpr (EXACT) {
                    const float4 d = *reinterpret_cast<const float4 *>(
                        reinterpret_cast<const float *>(w.rest + L::d) + (2 * bp + h) * kTile + ks * 16 + 4 * w.t);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float2 u = __fmul2_rn(make_float2(pe[n].x, pe[n].y), make_float2(d.x, d.y));
                        float2 v = __fmul2_rn(make_float2(pe[n].z, pe[n].w), make_float2(d.z, d.w));
                        if constexpr (EDGE) {
                            u.x = pe[n].x == 0.0f ? 0.0f : u.x;
                            u.y = pe[n].y == 0.0f ? 0.0f : u.y;
                            v.x = pe[n].z == 0.0f ? 0.0f : v.x;
                            v.y = pe[n].w == 0.0f ? 0.0f : v.y;
                        }
                        // odd columns: minus the first part
                        u = __fadd2_rn(u, make_float2(minus_part(u.x, keep), minus_part(u.y, keep)));
                        v = __fadd2_rn(v, make_float2(minus_part(v.x, keep), minus_part(v.y, keep)));
                        b0[n] = pack_rz(u.x, u.y);
                        b1[n] = pack_rz(v.x, v.y);
                    }
                } else {
                    const uint2 d = *reinterpret_cast<const uint2 *>(
                        reinterpret_cast<const uint32_t *>(w.rest + L::d) + (2 * bp + h) * (kTile / 2) + ks * 8 + 2 * w.t);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        b0[n] = hmul2(pw[n][ks][0], d.x);
                        b1[n] = hmul2(pw[n][ks][1], d.y);
                        if constexpr (EDGE) {
                            b0[n] &= not_zero2(pw[n][ks][0]);
                            b1[n] &= not_zero2(pw[n][ks][1]);
                        }
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float (&a0)[4] = acc[n][h][0], (&a1)[4] = acc[n][h][1];
                    if (ks == 0) {
                        mma16816(a0, xa, xb, ya, yb, b0[n], b1[n], 0.0f, 0.0f, 0.0f, 0.0f);
                        mma16816(a1, xc, xd, yc, yd, b0[n], b1[n], 0.0f, 0.0f, 0.0f, 0.0f);
                    } else {
                        mma16816(a0, xa, xb, ya, yb, b0[n], b1[n], a0[0], a0[1], a0[2], a0[3]);
                        mma16816(a1, xc, xd, yc, yd, b0[n], b1[n], a1[0], a1[1], a1[2], a1[3]);
                    }
                }
            }
        }
        const float2 units = unit[bp];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float2 f2 = make_float2(f[n][0], f[n][EXACT ? 0 : 1]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float u = h ? units.y : units.x;
                const float2 g2 = make_float2(g[n][0] * u, g[n][EXACT ? 0 : 1] * u);
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 v = make_float2(acc[n][h][m][2 * i], acc[n][h][m][2 * i + 1]);
                        w.out[n][2 * bp + h][m][i] = __ffma2_rn(w.out[n][2 * bp + h][m][i], f2, __fmul2_rn(v, g2));
                    }
            }
        }
    }
}

// Tiles [t0, t1) of an item.
template <int D, int NT, bool EXACT>
__device__ __forceinline__ void run_part(const StreamParams &p, WarpState<D, NT, EXACT> &w, Part &part,
                                         const Request &r, const Item &it, int t0, int t1) {
    using L = Layout<D, NT, EXACT>;
    constexpr int NB = L::NB, R = WarpState<D, NT, EXACT>::R;
    const AttnArgs &a = p.a;
    const float ninf = __uint_as_float(0xFF800000u);
    // the weights' largest value, and the least that goes with it in one pass
    constexpr float kFull = EXACT ? 1.0f : 16384.0f, kLow = kFull * kFaint, kRaise = 14.0f;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int k = 0; k < R; ++k) {
            w.top[n][k] = ninf;
            w.sum[n][k] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < NB * 4; ++i) w.out[n][i >> 2][(i >> 1) & 1][i & 1] = make_float2(0.0f, 0.0f);
    }
    // page indices of the keys ahead
    Pages pages = {-1, -64};
    auto ahead = [&](int key0) {  // makes the pages of the tile at key0 known
        const int first = key0 >> p.page_shift;
        if (first + max(1, kTile >> p.page_shift) > pages.first + 32) {
            pages.first = first;
            pages.lane_page =
                first + w.lane < a.table_width ? a.table[part.b * a.table_width + first + w.lane] : -1;
        }
    };
    const uint32_t codes_at = smem_addr(w.codes), scales_at = smem_addr(w.rest);
    auto fetch_k = [&](int key0) {
        fetch_tile<D>(p, p.k_codes, p.k_scales, codes_at, scales_at, part.to.kv_head, key0, part.lo, part.hi, pages,
                      w.lane);
    };
    auto fetch_v = [&](int key0) {
        fetch_tile<D>(p, p.v_codes, p.v_scales, codes_at + L::codes, scales_at + L::v_scales, part.to.kv_head, key0,
                      part.lo, part.hi, pages, w.lane);
    };
    int key0, end;
    {
        // the keys that any, and that every, row of the group sees
        const int heads = a.heads / p.kv_heads, all = r.rows * heads;
        const int pos0 = r.first + it.group * L::rows / heads;
        const int pos1 = r.first + (min((it.group + 1) * L::rows, all) - 1) / heads;
        const int lo = first_key(a, pos0), hi = a.causal ? min(r.len, pos1 + 1) : r.len;
        key0 = max((r.tile0 + t0) * kTile, lo / kTile * kTile);
        end = min((r.tile0 + t1) * kTile, hi);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < R; ++k) w.unit[n][k] = 1.0f;
        if (w.lane == 0) {
            part.b = it.b;
            part.lo = lo;
            part.hi = hi;
            part.lo_all = first_key(a, pos1);
            part.hi_all = a.causal ? min(r.len, pos0 + 1) : r.len;
        }
        __syncwarp();
        if (key0 < end) {
            QueryRows<D, NT, EXACT> rows;
            ahead(key0);
            load_q(p, rows, r, it, w.lane);  // under way while the pages are looked up
            fetch_k(key0);
            fetch_v(key0);
            stage_q(p, w, rows, part, r, all - it.group * L::rows);
        }
    }
    for (; key0 < end; key0 += kTile) {
        // 16-key groups whose page can be read: lane i looks at group i
        const int32_t page = __shfl_sync(0xFFFFFFFFu, pages.lane_page,
                                         (((key0 + 16 * w.lane) >> p.page_shift) - pages.first) & 31);
        const int key = key0 + 16 * w.lane;
        const unsigned lost = __ballot_sync(0xFFFFFFFFu, w.lane < 4 && key < part.hi && key + 16 > part.lo &&
                                                             (page < 0 || page >= p.num_pages));
        if (lost && w.lane == 0) record_error(p.ctx, kDevErrIndex);
        const bool edge = lost || key0 < part.lo_all || key0 + kTile > part.hi_all;

        copies_wait();  // K is there; V may be under way
        float s[NT][4][R][2];
        tile_scores<D, NT, EXACT>(w, p.magic, s);
        __syncwarp();
        if (key0 + kTile < end) {
            ahead(key0 + kTile);
            fetch_k(key0 + kTile);
        } else {
            copies_commit();
        }
        unsigned seen = 3u;  // keys 2 lane and 2 lane + 1, by any row
        if (edge) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int k = 0; k < R; ++k) {
                        const int row = EXACT ? n * 4 + w.t : n * 8 + 2 * w.t + k;
                        const int row_lo = part.row_lo[row], row_hi = part.row_hi[row];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int j = key0 + 16 * m + 8 * h + w.g;
                            if (j < row_lo || j >= row_hi || ((lost >> m) & 1u)) s[n][m][k][h] = ninf;
                        }
                    }
            const int j = key0 + 2 * w.lane, lo = part.lo, hi = part.hi;
            seen = (lost >> (w.lane >> 3)) & 1u ? 0u : (j >= lo && j < hi ? 1u : 0u) | (j + 1 >= lo && j + 1 < hi ? 2u : 0u);
        }
        // the rows' largest and smallest scores of the tile
        float top[NT][R];
        bool faint = false;  // some weight lies below 2^-24 of the tile's largest
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < R; ++k) {
                float v = s[n][0][k][0], u = v;
#pragma unroll
                for (int i = 1; i < 8; ++i) {
                    v = fmaxf(v, s[n][i >> 1][k][i & 1]);
                    u = fminf(u, s[n][i >> 1][k][i & 1]);
                }
                v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 4));
                v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 8));
                v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 16));
                top[n][k] = v * w.unit[n][k];
                faint |= u * w.unit[n][k] < top[n][k] - 23.5f;
            }
        copies_wait();  // V is there; the next K may be under way
        tile_scales<D, NT, EXACT>(w, seen);
        // f: factor of what is there already; g: of this tile's products.  The
        // products carry 2^14 of the scales (bf16 output: of the weights) and, for
        // bf16 output, 2^-24 of the codes, beside their block's unit.
        float f[NT][R], g[NT][R];
        float *pp = reinterpret_cast<float *>(w.rest + L::p) + (w.g >> 1) * 4 + (w.g & 1);
        uint32_t pw[NT][4][2];
        const float unit_out = pow2i(EXACT ? -14 : 10);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int k = 0; k < R; ++k) {
                const float here = top[n][k] == ninf ? 0.0f : top[n][k], now = fmaxf(w.top[n][k], top[n][k]);
                f[n][k] = w.top[n][k] == ninf ? 0.0f : exp2_fast(w.top[n][k] - now);
                const float fresh = top[n][k] == ninf ? 0.0f : exp2_fast(top[n][k] - now);
                g[n][k] = fresh * unit_out;
                w.top[n][k] = now;
                // bf16 output: raised by 2^14 as the B operand takes them
                const float base = EXACT ? -here : kRaise - here;
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float e = exp2_fast(fmaf(s[n][i >> 1][k][i & 1], w.unit[n][k], base));
                    s[n][i >> 1][k][i & 1] = e;
                    sum += e;
                }
                w.sum[n][k] = fmaf(w.sum[n][k], f[n][k], sum * (EXACT ? fresh : fresh * (1.0f / 16384.0f)));
            }
        }
        if (__any_sync(0xFFFFFFFFu, faint)) {  // hidden keys, whose weight is 0, do not count
            faint = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < R; ++k)
#pragma unroll
                    for (int i = 0; i < 8; ++i) faint |= s[n][i >> 1][k][i & 1] < kLow && s[n][i >> 1][k][i & 1] > 0.0f;
            faint = __any_sync(0xFFFFFFFFu, faint);
        }
        // the weights as the B operand's keys and columns
        auto hand_over = [&](auto pick) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if constexpr (EXACT) {
                            pp[(n * 4 + w.t) * L::p_stride + 16 * m + 2 * h] = pick(s[n][m][0][h]);
                        } else {
                            pw[n][m][h] = transpose8(pack_rn(pick(s[n][m][0][h]), pick(s[n][m][R - 1][h])));
                        }
                    }
            __syncwarp();
        };
        // Weights far below the tile's largest would fall out of binary16's
        // range, which shows where the large ones meet zeros: they go in
        // passes of their own, raised by 2^24 each time.
        if (faint) {
            for (float raise = 1.0f / kFaint; faint; raise *= 1.0f / kFaint) {
                bool more = false;
                float low[NT][R];  // factor of the pass's products
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int k = 0; k < R; ++k) {
                        low[n][k] = g[n][k] / raise;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float e = s[n][i >> 1][k][i & 1] * raise;
                            more |= e < kLow && e > 0.0f;
                        }
                    }
                hand_over([raise](float v) {
                    const float e = v * raise;
                    return e >= kLow && e < kFull ? e : 0.0f;
                });
                tile_values<D, NT, EXACT, true>(w, p.magic, pw, f, low);
                __syncwarp();
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int k = 0; k < R; ++k) f[n][k] = 1.0f;
                faint = __any_sync(0xFFFFFFFFu, more);
            }
            hand_over([](float e) { return e < kLow ? 0.0f : e; });
        } else {
            hand_over([](float e) { return e; });
        }
        if (edge)
            tile_values<D, NT, EXACT, true>(w, p.magic, pw, f, g);
        else
            tile_values<D, NT, EXACT, false>(w, p.magic, pw, f, g);
        __syncwarp();
        if (key0 + kTile < end) fetch_v(key0 + kTile);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < R; ++k) {
            w.sum[n][k] += __shfl_xor_sync(0xFFFFFFFFu, w.sum[n][k], 4);
            w.sum[n][k] += __shfl_xor_sync(0xFFFFFFFFu, w.sum[n][k], 8);
            w.sum[n][k] += __shfl_xor_sync(0xFFFFFFFFu, w.sum[n][k], 16);
        }
}

// The lane's accumulators as outputs, unnormalised, row by row: begin(n, k,
// row) returns a function of (dimension, value).
template <int D, int NT, bool EXACT, typename Begin>
__device__ __forceinline__ void each_output(const WarpState<D, NT, EXACT> &w, int rows, Begin begin) {
    constexpr int NB = D / 32, R = WarpState<D, NT, EXACT>::R;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int row = EXACT ? n * 4 + w.t : n * 8 + 2 * w.t + k;
            if (row >= rows) continue;
            auto put = begin(n, k, row);
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float2 o = w.out[n][b][m][h];
                        const float v = EXACT ? o.x + o.y : k ? o.y : o.x;
                        put(32 * b + 16 * h + 2 * w.g + m, v * (!EXACT && h ? 0.0625f : 1.0f));
                    }
        }
}

// How many rows an item has.
template <int ROWS>
__device__ __forceinline__ int rows_of(const StreamParams &p, const Target &to) {
    return min(ROWS, to.rows * (p.a.heads / p.kv_heads) - to.group * ROWS);
}

// The row of q, and the head, that row `row` of an item stands for; false for
// rows past the request's last.
template <int ROWS>
__device__ __forceinline__ bool locate(const StreamParams &p, const Target &to, int row, int64_t &at, int &head) {
    const int heads = p.a.heads / p.kv_heads, flat = to.group * ROWS + row;
    if (flat >= to.rows * heads) return false;
    const int token = flat / heads;
    head = to.kv_head * heads + flat - token * heads;
    at = static_cast<int64_t>(to.row0) + token;
    return true;
}

// Four consecutive outputs of an item's row, from their weighted sums.
template <int D, int ROWS>
__device__ __forceinline__ void write_out(const StreamParams &p, const Target &to, int row, int d, const float4 &v,
                                          float sum) {
    int64_t at;
    int head;
    if (!locate<ROWS>(p, to, row, at, head)) return;
    at = at * p.a.out_stride + static_cast<int64_t>(head) * D + d;
    const float down = sum == 0.0f ? 0.0f : 1.0f / sum;
    store_value(p.a.out, at, p.a.out_bf16, v.x * down);
    store_value(p.a.out, at + 1, p.a.out_bf16, v.y * down);
    store_value(p.a.out, at + 2, p.a.out_bf16, v.z * down);
    store_value(p.a.out, at + 3, p.a.out_bf16, v.w * down);
}

template <int ROWS>
__device__ __forceinline__ void write_lse(const StreamParams &p, const Target &to, int row, float top, float sum) {
    int64_t at;
    int head;
    if (p.a.lse && locate<ROWS>(p, to, row, at, head))
        p.a.lse[at * p.a.heads + head] = sum == 0.0f ? __uint_as_float(0xFF800000u) : (top + log2f(sum)) * kLn2;
}

template <int D, int NT, bool EXACT>
__global__ void __launch_bounds__((Layout<D, NT, EXACT>::threads), (Layout<D, NT, EXACT>::ctas))
    attn_stream_kernel(const __grid_constant__ StreamParams p) {
    using L = Layout<D, NT, EXACT>;
    constexpr int R = WarpState<D, NT, EXACT>::R, ROWS = L::rows, W = L::warps;
    extern __shared__ uint8_t attn_smem[];
    uint8_t *base = attn_smem + ((1024u - (smem_addr(attn_smem) & 1023u)) & 1023u);
    Shared &sh = *reinterpret_cast<Shared *>(base + W * (L::code_bytes + L::rest_bytes));
    const int warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_launch_dependents();
    const Line line = build_line<ROWS, W>(p, sh);

    WarpState<D, NT, EXACT> w;
    w.codes = base + warp * L::code_bytes;
    w.rest = base + W * L::code_bytes + warp * L::rest_bytes;
    w.lane = threadIdx.x & 31;
    w.g = w.lane >> 2;
    w.t = w.lane & 3;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * W;
    const int64_t me = static_cast<int64_t>(blockIdx.x) * W + warp;
    // equal shares of the line, or one place each
    const int64_t share = line.total / warps, left = line.total - share * warps;
    const int64_t x0 = line.spread ? min(me, line.total) : share * me + min(me, left);
    const int64_t x1 = line.spread ? min(me + 1, line.total) : x0 + share + (me < left ? 1 : 0);
    Part &part = sh.part[warp];
    if (w.lane == 0) {
        sh.flags[warp] = kEmpty;
        part.x = x0;
        part.end = x1;
    }
    __syncwarp();
    while (part.x < part.end) {
        {
            const int64_t x = part.x;
            int64_t before;
            Request r;
            Item it;
            it.b = find_request<ROWS, W>(p, sh, line, x, before, r);
            const int places = item_places<W>(r, line.spread);
            // most offsets fit 32 bits, whose division is far cheaper
            const int64_t off = x - before;
            const int item = off <= INT32_MAX ? static_cast<int>(off) / places : static_cast<int>(off / places);
            it.kv_head = item / r.groups;
            it.group = item - it.kv_head * r.groups;
            const int t0 = static_cast<int>(off - static_cast<int64_t>(item) * places);
            if (t0 >= r.tiles) break;  // a place without a tile (spread: the warp's only one)
            const int t1 = static_cast<int>(min(static_cast<int64_t>(r.tiles), t0 + (part.end - x)));
            __syncwarp();
            if (w.lane == 0) {
                part.x = x + t1 - t0;
                part.t0 = t0;
                part.t1 = t1;
                part.tiles = r.tiles;
                part.to = Target{r.row0, r.rows, it.kv_head, it.group};
            }
            run_part<D, NT, EXACT>(p, w, part, r, it, t0, t1);
            __syncwarp();
        }
        const Target to = part.to;
        const int rows = rows_of<ROWS>(p, to);
        if (part.t0 == 0 && part.t1 == part.tiles) {
            each_output<D, NT, EXACT>(w, rows, [&](int n, int k, int row) {
                int64_t at = 0;
                int head = 0;
                locate<ROWS>(p, to, row, at, head);
                at = at * p.a.out_stride + static_cast<int64_t>(head) * D;
                const float down = w.sum[n][k] == 0.0f ? 0.0f : 1.0f / w.sum[n][k];
                return [&p, at, down](int d, float v) { store_value(p.a.out, at + d, p.a.out_bf16, v * down); };
            });
            if (w.g == 0)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int k = 0; k < R; ++k)
                        write_lse<ROWS>(p, to, EXACT ? n * 4 + w.t : n * 8 + 2 * w.t + k, w.top[n][k], w.sum[n][k]);
            if (w.lane == 0) sh.flags[warp] &= ~kEmpty;
            __syncwarp();
            continue;
        }
        // the warp's last part stays in its code buffers, which no later tile
        // needs; an earlier one goes to global memory
        const bool head = part.t0 > 0, last = part.x >= part.end;
        float *rec = last ? reinterpret_cast<float *>(w.codes)
                          : p.warp_records + (static_cast<int64_t>(blockIdx.x) * W + warp) * kRecord;
        each_output<D, NT, EXACT>(w, rows, [rec](int, int, int row) { return [=](int d, float v) { rec[row * D + d] = v; }; });
        if (w.g == 0)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    float *s = sh.stat[warp][head ? 0 : 1][EXACT ? n * 4 + w.t : n * 8 + 2 * w.t + k];
                    s[0] = w.top[n][k];
                    s[1] = w.sum[n][k];
                }
        if (w.lane == 0) {
            sh.target[warp][head ? 0 : 1] = to;
            sh.flags[warp] = (sh.flags[warp] & ~kEmpty) |
                             (head ? kHead | (part.t1 < part.tiles ? kHeadOpen : 0) | (last ? kHeadLast : 0) : kTail);
        }
        __syncwarp();
    }
    __syncthreads();

    // Join the warps' parts.  A chain begins with a tail, or with the head of
    // the first warp that has tiles, and goes on over heads while they are
    // open; empty warps may lie between.
    CtaParts mine = {kEmpty, {}};
    for (int c = 0; c < W; ++c) {
        const int fc = sh.flags[c];
        if (fc & kEmpty) continue;
        const bool first = mine.flags == kEmpty;
        if (first) mine.flags = 0;
        for (int kind = first && (fc & kHead) ? 0 : 1; kind < 2; ++kind) {
            if (kind == 1 && !(fc & kTail)) continue;
            bool open = kind == 1 || (fc & kHeadOpen);
            unsigned members = 0;
            for (int j = c + 1; j < W && open; ++j) {
                if (sh.flags[j] & kEmpty) continue;
                members |= 1u << j;
                open = sh.flags[j] & kHeadOpen;
            }
            const Target to = sh.target[c][kind];
            const bool whole = kind == 1 && !open;
            float *dst = p.cta_records + (static_cast<int64_t>(blockIdx.x) * 2 + kind) * kRecord;
            if (threadIdx.x < ROWS * kWarps) {  // weights of the parts, eight lanes a row
                const int row = threadIdx.x / kWarps, j = threadIdx.x % kWarps;
                const bool member = j < W && (j == c || (j > c && ((members >> j) & 1u)));
                const float *st = sh.stat[member ? j : c][member && j > c ? 0 : kind][row];
                float top = st[0];
#pragma unroll
                for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                const float ref = top == __uint_as_float(0xFF800000u) ? 0.0f : top;
                const float f = member ? exp2_fast(st[0] - ref) : 0.0f;
                float sum = member ? f * st[1] : 0.0f;
#pragma unroll
                for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
                sh.weight[row][j] = f;
                if (j == 0) {
                    sh.total[row][0] = top;
                    sh.total[row][1] = sum;
                    if (whole)
                        write_lse<ROWS>(p, to, row, top, sum);
                    else
                        *reinterpret_cast<float2 *>(dst + kRecordStat + 2 * row) = make_float2(top, sum);
                }
            }
            __syncthreads();
            for (int i = threadIdx.x; i < rows_of<ROWS>(p, to) * (D / 4); i += L::threads) {
                const int row = i / (D / 4), d = (i - row * (D / 4)) * 4;
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    if (j != c && !((members >> j) & 1u)) continue;
                    const bool inside = (j == c && kind == 1) || (sh.flags[j] & kHeadLast);
                    const float *rec = inside ? reinterpret_cast<const float *>(base + j * L::code_bytes)
                                              : p.warp_records + (static_cast<int64_t>(blockIdx.x) * W + j) * kRecord;
                    const float4 x = *reinterpret_cast<const float4 *>(rec + i * 4);
                    const float f = sh.weight[row][j];
                    v.x = fmaf(f, x.x, v.x);
                    v.y = fmaf(f, x.y, v.y);
                    v.z = fmaf(f, x.z, v.z);
                    v.w = fmaf(f, x.w, v.w);
                }
                if (whole)
                    write_out<D, ROWS>(p, to, row, d, v, sh.total[row][1]);
                else
                    *reinterpret_cast<float4 *>(dst + i * 4) = v;
            }
            __syncthreads();
            if (!whole) {
                if (kind == 0) {
                    mine.flags |= kHead | (open ? kHeadOpen : 0);
                } else {
                    mine.flags |= kTail;
                    mine.target = to;
                }
            }
        }
    }
    if (threadIdx.x == 0) p.parts[blockIdx.x] = mine;
}

// Joins the items that several CTAs hold: CTA x of this grid the one that CTA
// x's tail begins, 128 outputs of it per y.  The eight warps take every eighth
// part each, a lane four outputs of it.
constexpr int kMaxCtas = 512;
constexpr int kJoinOutputs = 128;

template <int D, int ROWS>
__global__ void __launch_bounds__(kThreads) attn_join_kernel(const StreamParams p) {
    constexpr int RB = D < kJoinOutputs ? kJoinOutputs / D : 1;  // rows of a CTA
    __shared__ int flags[kMaxCtas];
    __shared__ int list[kMaxCtas];
    __shared__ int count;
    __shared__ float weight[RB][kMaxCtas];
    __shared__ float total[RB][2];
    __shared__ float4 share[kWarps][32];
    pdl_wait();
    pdl_launch_dependents();
    const int n = gridDim.x, c = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const CtaParts mine = p.parts[c];
    if (!(mine.flags & kTail) || static_cast<int>(blockIdx.y) * kJoinOutputs >= rows_of<ROWS>(p, mine.target) * D) return;
    for (int i = threadIdx.x; i < n; i += kThreads) flags[i] = p.parts[i].flags;
    __syncthreads();
    if (warp == 0) {  // the parts: c's tail, then heads up to the first that is not open
        int k = 1;
        if (lane == 0) list[0] = c;
        for (int i = c + 1; i < n; i += 32) {
            const int f = i + lane < n ? flags[i + lane] : kEmpty;
            const bool there = !(f & kEmpty), ends = there && !(f & kHeadOpen);
            const unsigned stop = __ballot_sync(0xFFFFFFFFu, ends);
            const unsigned upto = stop ? (stop & -stop) * 2u - 1u : 0xFFFFFFFFu;  // lanes up to the first that ends
            const unsigned take = __ballot_sync(0xFFFFFFFFu, there) & upto;
            if ((take >> lane) & 1u) list[k + __popc(take & ((1u << lane) - 1u))] = i + lane;
            k += __popc(take);
            if (stop) break;
        }
        if (lane == 0) count = k;
    }
    __syncthreads();
    const int k = count, first = blockIdx.y * kJoinOutputs;
    auto record = [&](int i) { return p.cta_records + (static_cast<int64_t>(list[i]) * 2 + (i == 0 ? 1 : 0)) * kRecord; };
    if (warp < RB) {  // the weights of one row
        const int row = first / D + warp;
        const float ninf = __uint_as_float(0xFF800000u);
        float top = ninf;
        for (int i = lane; i < k; i += 32) {
            const float t = record(i)[kRecordStat + 2 * row];
            weight[warp][i] = t;
            top = fmaxf(top, t);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        const float ref = top == ninf ? 0.0f : top;
        float sum = 0.0f;
        for (int i = lane; i < k; i += 32) {
            const float f = exp2_fast(weight[warp][i] - ref);
            weight[warp][i] = f;
            sum = fmaf(f, record(i)[kRecordStat + 2 * row + 1], sum);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if (lane == 0) {
            total[warp][0] = top;
            total[warp][1] = sum;
        }
    }
    __syncthreads();
    const int at = first + lane * 4, sub = at / D - first / D;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int i = warp; i < k; i += kWarps) {
        const float4 x = *reinterpret_cast<const float4 *>(record(i) + at);
        const float f = weight[sub][i];
        v.x = fmaf(f, x.x, v.x);
        v.y = fmaf(f, x.y, v.y);
        v.z = fmaf(f, x.z, v.z);
        v.w = fmaf(f, x.w, v.w);
    }
    share[warp][lane] = v;
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int j = 1; j < kWarps; ++j) {
        const float4 x = share[j][lane];
        v.x += x.x;
        v.y += x.y;
        v.z += x.z;
        v.w += x.w;
    }
    const int row = at / D, d = at - row * D;
    write_out<D, ROWS>(p, mine.target, row, d, v, total[sub][1]);
    if (d == 0) write_lse<ROWS>(p, mine.target, row, total[sub][0], total[sub][1]);
}

template <int D, int NT, bool EXACT>
cudaError_t launch_stream(const KvCache &c, const AttnArgs &a, cudaStream_t stream, const LaunchCtx &ctx) {
    using L = Layout<D, NT, EXACT>;
    static int limits[kMaxDevices];
    constexpr size_t smem = static_cast<size_t>(L::warps) * (L::code_bytes + L::rest_bytes) + sizeof(Shared) + 1024;
    static_assert(sizeof(Shared) <= 14336 && smem <= 232448, "shared memory per CTA");
    auto *kernel = attn_stream_kernel<D, NT, EXACT>;
    cudaError_t e = ensure_smem(kernel, smem, false, limits);
    if (e != cudaSuccess) return e;
    const int ctas = std::min(device_sm_count() * L::ctas, kMaxCtas);
    StreamParams p = {};
    p.a = a;
    p.k_codes = static_cast<const uint8_t *>(c.k_codes);
    p.k_scales = static_cast<const uint8_t *>(c.k_scales);
    p.v_codes = static_cast<const uint8_t *>(c.v_codes);
    p.v_scales = static_cast<const uint8_t *>(c.v_scales);
    p.num_pages = static_cast<int>(c.num_pages);
    p.page_shift = c.page_shift;
    p.kv_heads = c.kv_heads;
    p.q_pairs = a.q_stride % 2 == 0 && reinterpret_cast<uintptr_t>(a.q) % (a.q_bf16 ? 4 : 8) == 0;
    p.magic = 0x64006400u;
    p.warp_records = static_cast<float *>(a.workspace);
    p.cta_records = p.warp_records + static_cast<size_t>(ctas) * kWarps * kRecord;
    p.parts = reinterpret_cast<CtaParts *>(p.cta_records + static_cast<size_t>(ctas) * 2 * kRecord);
    p.ctx = ctx;
    e = launch_kernel(kernel, dim3(ctas), dim3(L::threads), smem, stream, 1, p);
    if (e != cudaSuccess) return e;
    return launch_kernel(attn_join_kernel<D, L::rows>, dim3(ctas, L::rows * D / kJoinOutputs), dim3(kThreads), 0, stream,
                         1, p);
}

template <int D>
cudaError_t launch_dim(const KvCache &c, const AttnArgs &a, cudaStream_t stream, const LaunchCtx &ctx) {
    if (a.out_bf16) return launch_stream<D, 1, false>(c, a, stream, ctx);
    // Four rows fill a column tile; two tiles share the codes' work, but take
    // registers from the overlap of tiles.  Us per call with one / two, two
    // key heads: head_dim 128, 16 requests of 4000 keys: 2 rows 15 / 17, 16
    // rows 28 / 27; 32 rows of one with 16000 keys 22 / 21, 256 rows 76 / 61,
    // 2048 rows 499 / 350; head_dim 64, 16 rows 20 / 23, 256 rows 47 / 45, 2048
    // rows 266 / 214.  head_dim 256, where two tiles' outputs are 256
    // registers: 4 rows 17 / 26, 8 rows 28 / 43, 256 rows 134 / 146, 2048 rows
    // 933 / 999.
    if constexpr (D < 256)
        if (static_cast<int64_t>(a.max_q) * (a.heads / c.kv_heads) >= 32) return launch_stream<D, 2, true>(c, a, stream, ctx);
    return launch_stream<D, 1, true>(c, a, stream, ctx);
}

}  // namespace

size_t attn_workspace_bytes(const KvCache &, int) {
    const size_t ctas = std::min(device_sm_count() * 2, kMaxCtas);  // as the smaller head dimensions take
    return std::max(ctas * ((kWarps + 2) * kRecord * sizeof(float) + sizeof(CtaParts)), attn_tiles_workspace_bytes());
}

cudaError_t launch_attn(const KvCache &c, const AttnArgs &a, cudaStream_t stream, const LaunchCtx &ctx) {
    if (attn_tiles_pay(c, a)) return launch_attn_tiles(c, a, stream, ctx);
    if (c.head_dim == 64) return launch_dim<64>(c, a, stream, ctx);
    if (c.head_dim == 128) return launch_dim<128>(c, a, stream, ctx);
    return launch_dim<256>(c, a, stream, ctx);
}

}  // namespace qmm
