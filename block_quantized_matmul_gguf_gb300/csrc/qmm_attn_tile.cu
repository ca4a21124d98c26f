// qmm_attn_tile.cu -- attention over the paged Q4_0 cache on the tcgen05
// tensor cores, for the prompts' many query rows (bf16 output).
//
// One CTA takes 128 query rows (head_dim 256) or 256 (64, 128) of one request
// and key head -- the query heads of a group side by side -- over their keys,
// or a part of them where the blocks are too few for the GPU, in tiles of 64:
//   S = Q K^T    M = 128 rows, N = 64 keys, K = head_dim; Q in tensor memory
//   P = 2^(S - m) in binary16, written over S
//   O += P V     M = 128 rows, N = head_dim, K = 64 keys; O in tensor memory
// Warps by role:
//   softmax   4 per 128 rows, a thread per row: stages Q, turns S into P,
//             keeps maximum and sum, scales O when the maximum has grown by
//             more than kSlack powers of two, writes the output
//   dequant   8: codes and scales from global memory (plain loads: an append
//             may write them until pdl_wait), a tile ahead in registers, to
//             binary16 rows of 64 values with the 128-byte swizzle; K is then a
//             K-major operand and V, its rows being keys too, an MN-major one
//             of the same layout
//   MMA       one per 128 rows; S of the next tile is formed while a tile is
//             in the softmax (head_dim 256), or the other rows' products run
// Values keep the order in which a word of codes gives them (0 2 16 18 1 3 17
// 19 and so on); Q is staged in that order and the outputs are put back.
//
// Precision: q, (n - 8) d and the weights are rounded once to binary16 each.
// K and V are scaled by powers of two, one for the keys of each dequant warp,
// to below 2^-6 (16 where the scales lie far apart), q per row to below 2^15
// and the weights to at most 2^15, so that nothing overflows.  Weights below
// 2^-24 of a row's reference lose bits, or all of them, among binary16's
// subnormal numbers.  That shows only where the heavy keys leave (nearly)
// nothing of an output, whose size does not tell whether they cancel or are 0
// there.  A block with such a row goes over its tiles once more, by the same
// steps, with what was lost of the weights raised by 2^38, and adds the
// products; four passes cover fp32's range.  Dimensions in which every value
// is 0 do not count.  The case of 2048 tokens below by the scores' standard
// deviation, from a flushed L2: 1.2 198 us, 2.4 410, 4 435, 8 448, 24 714; with
// one block of values that are all 0 196, 427, 465, 482, 712.
//
// Parts are joined by a second kernel: their outputs and sums, in fp32, are
// weighted by 2^(m - largest m), in the parts' order.
//
// Bound by the chain of a tile's steps, which the two buffers of S overlap in
// part: at head_dim 256 a tile takes 2400 cycles, its dequantisation 2200
// (eight warps, two an SM quarter, that fill 64 KB of shared memory), its
// softmax 1600, its products 1290 (48 cycles for 64 columns and 130 for 256,
// as measured alone).  Measured: 2048 tokens of 8 heads of 256 (2 key heads)
// behind 6000 cached ones 168 us, 700 TFLOP/s; seven prompts of up to 700
// tokens of 16 heads of 128 with a window of 1024 keys 92 us; 128 tokens of
// the first layout behind 32000 75 us (777 with one CTA a block).
#include "qmm_attn.cuh"
#include "qmm_tc.cuh"

#include <algorithm>
#include <type_traits>

namespace qmm {
namespace {

constexpr int kKeys = 64;                  // of a tile
constexpr int kDequantWarps = 8;
constexpr int kRing = 16;                  // tiles whose exponents are kept
constexpr int kPanel = kKeys * 128;        // bytes of 64 values of a tile's keys
constexpr int kRaise = 10;                 // the reference weight is 2^10
constexpr float kSlack = 5.0f;             // ... and the largest at most 2^15
constexpr int kPasses = 4;                 // over a block's tiles, at most
constexpr float kNormal = 1.0f / 16384.0f; // binary16's smallest normal number
constexpr int kPassRaise = 38;             // what a pass loses of a weight (at most 2^-25) is raised to 2^13

template <int D>
struct Tile {
    static constexpr int QT = D == 256 ? 1 : 2;  // 128-row tiles; O of both fits tensor memory
    static constexpr int rows = 128 * QT;
    static constexpr int stages = D == 256 ? 3 : 4;
    static constexpr int bytes = kKeys * D * 2;
    static constexpr int softmax_warps = 4 * QT;
    static constexpr int mma_warp = softmax_warps + kDequantWarps;
    static constexpr int threads = (mma_warp + 4) * 32;  // whole warpgroups: the last warps only hold registers
    // registers of a thread: at launch, and by role (at most as many in all:
    // 512 x 128 >= 128 x (208 + 2 x 104 + 56), 640 x 96 >= 128 x (2 x 144 + 2 x 72 + 40))
    static constexpr int launch_regs = D == 256 ? 128 : 96;
    static constexpr int softmax_regs = D == 256 ? 208 : 144;
    static constexpr int dequant_regs = D == 256 ? 104 : 72;
    static constexpr int mma_regs = D == 256 ? 56 : 40;
    static_assert(softmax_warps * softmax_regs + kDequantWarps * dequant_regs + 4 * mma_regs <= threads / 32 * launch_regs,
                  "more registers than the block was launched with would be waited for in vain");
    static constexpr int units = D == 256 ? 2 : 1;  // blocks of 32 values per dequant thread
    // tensor memory columns
    static constexpr int o_col = 0, q_col = QT * D, s_col = q_col + QT * D / 2;
    static constexpr uint32_t tmem_cols = 512;
    static_assert(s_col + 2 * kKeys <= 512, "tensor memory");
    // S buffer of tile t for row tile qt (two in all), and the parity of its use
    static constexpr __host__ __device__ int buffer(int t, int qt) { return QT == 1 ? t & 1 : qt; }
    static constexpr __host__ __device__ uint32_t phase(int t) { return (QT == 1 ? t >> 1 : t) & 1; }
};

// What the softmax has to know of a tile, by groups of eight keys.
struct TileInfo {
    float k_unit[8];       // K of a group is scaled by 1 / k_unit
    int v_exp[8];          // V by 2^-(v_exp / 2); odd where its values may reach 16, not 2^-6
    uint32_t lost;         // 16-key groups without a page
    uint32_t pad[3];
};

// Rows of one request and key head, and the tiles of their keys: all, or a part.
struct Block {
    int b, kv_head;
    int q_row0, flat0, rows;       // first row of q of the request; first flat row, rows of the block
    int first, len;
    int lo, hi, lo_all, hi_all;    // keys that any, and that every, row sees
    int key0, tiles;
    int slot;                      // of a part in the workspace, or -1
};

// The parts of split blocks in the workspace, those of one block side by side.
struct TileParts {
    int count;        // first part of a block: its parts; else 0
    Block block;
};
struct TileHeader {
    int used;         // slots
    int pad[3];
};
constexpr int kMaxTileCtas = 256;  // SMs that are counted on: at most as many parts
constexpr int kMaxThreads = 640;
// Outputs of a part as float4 [rows / 8][D / 4][8 rows], then maximum and sum
// of each row.
constexpr int kPartFloats = 128 * 256 + 256 * 2;
constexpr int kMinPart = 8;  // tiles of a part at least: about what a CTA takes to begin and end

struct TileShared {
    uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
    uint64_t s_full[2], p_full[2], pv_done[2], final[2], q_ready;
    alignas(16) TileInfo info[kRing];
    int64_t scratch[32];
    int64_t blocks[kMaxThreads];  // row blocks before each thread's requests
    Block block;
    uint32_t tmem;
    int abort;
    int again[kPasses];             // whether another pass follows this one
    int odd;                        // whether some value's scale is a NaN or an infinity
    int any_zero;                   // whether sh.zero has a digit
    // by block, digits of V's codes: in which the outputs of a warp's rows are all
    // 0 that might have lost something, and of those, in which some value is not
    alignas(16) uint32_t zero[8][4], found[8][4];
};

struct TileParams {
    AttnArgs a;
    const uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
    int num_pages, page_shift, kv_heads;
    bool q_wide, out_wide;  // rows are 16-byte aligned
    int split;               // SMs to fill with parts of blocks, or 0: whole blocks only
    TileHeader *header;
    TileParts *parts;        // [slots]
    float *records;          // [slots][kPartFloats]
    LaunchCtx ctx;
};

// kind::f16 with binary16 operands and fp32 sums, M = 128; b_rows: B's rows
// are along K (MN-major).
constexpr uint32_t tile_idesc(int n, bool b_rows) {
    return (1u << 4) | (b_rows ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | ((128u >> 4) << 24);
}

// B operand with rows along K: 8-row groups 1024 bytes apart, 64-value panels
// kPanel bytes apart.
__device__ __forceinline__ uint64_t rows_desc(uint32_t saddr) {
    uint64_t d = static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(kPanel >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

// A warpgroup's registers per thread, from its launch's pool.
template <int N>
__device__ __forceinline__ void registers_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void registers_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// ---- which rows and keys this CTA takes ----------------------------------------------

template <int D>
__device__ __forceinline__ int request_blocks(const TileParams &p, const RequestRows &r) {
    return static_cast<int>((static_cast<int64_t>(r.rows) * (p.a.heads / p.kv_heads) + Tile<D>::rows - 1) / Tile<D>::rows);
}

template <int D>
__device__ __forceinline__ Block block_of(const TileParams &p, const RequestRows &r, int b, int at, int kv_head) {
    using T = Tile<D>;
    const int heads = p.a.heads / p.kv_heads;
    Block k;
    k.b = b;
    k.kv_head = kv_head;
    k.q_row0 = r.row0;
    k.flat0 = at * T::rows;
    k.rows = min(T::rows, r.rows * heads - k.flat0);
    k.first = r.first;
    k.len = r.len;
    const int pos0 = r.first + k.flat0 / heads, pos1 = r.first + (k.flat0 + k.rows - 1) / heads;
    k.lo = first_key(p.a, pos0);
    k.hi = p.a.causal ? min(r.len, pos1 + 1) : r.len;
    k.lo_all = first_key(p.a, pos1);
    k.hi_all = p.a.causal ? min(r.len, pos0 + 1) : r.len;
    k.key0 = k.lo / kKeys * kKeys;
    k.tiles = k.hi > k.lo ? (k.hi - k.key0 + kKeys - 1) / kKeys : 0;
    k.slot = -1;
    return k;
}

// The last thread whose count is at most x.
template <int THREADS>
__device__ __forceinline__ int holder(const int64_t *before, int64_t x) {
    int lo = 0, n = THREADS;
    while (n > 1) {
        const int half = n >> 1;
        if (before[lo + half] <= x) lo += half, n -= half;
        else n = half;
    }
    return lo;
}

// Row blocks one after another.
template <int D>
struct Walk {
    int b, at, n;  // request, row blocks of it that come before, its row blocks
    RequestRows r;
    // the last rows see the most keys: they go first
    __device__ __forceinline__ Block block(const TileParams &p, int kv_head) const { return block_of<D>(p, r, b, n - 1 - at, kv_head); }
    __device__ __forceinline__ void start(const TileParams &p, const TileShared &sh, int64_t block) {
        constexpr int threads = Tile<D>::threads;
        const int t = holder<threads>(sh.blocks, block);
        b = t * ((p.a.batch + threads - 1) / threads);
        int64_t left = block - sh.blocks[t];
        for (;; ++b) {
            r = request_rows(p.a, p.page_shift, b);
            n = request_blocks<D>(p, r);
            if (left < n || b + 1 >= p.a.batch) break;
            left -= n;
        }
        at = static_cast<int>(left);
    }
    __device__ __forceinline__ void next(const TileParams &p) {
        ++at;
        while (at >= n && b + 1 < p.a.batch) {
            r = request_rows(p.a, p.page_shift, ++b);
            n = request_blocks<D>(p, r);
            at = 0;
        }
    }
};

// Exclusive sum over the CTA's threads, and the total.
template <int THREADS>
__device__ __forceinline__ int64_t sum_before(TileShared &sh, int64_t mine, int64_t &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xFFFFFFFFu, sum, o);
        if (lane >= o) sum += up;
    }
    if (lane == 31) sh.scratch[warp] = sum;
    __syncthreads();
    int64_t before = sum - mine;
    total = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += sh.scratch[w];
        total += sh.scratch[w];
    }
    __syncthreads();
    return before;
}

// Fills sh.block; block.b is -1 for CTAs past the last.
// Split, a block of more than so many tiles is cut into equal parts for CTAs
// of their own: all parts run at once where the blocks are fewer than 3/4 of
// the SMs, and otherwise none has more than two SMs' share of the work.
template <int D>
__device__ __forceinline__ void find_block(const TileParams &p, TileShared &sh) {
    constexpr int threads = Tile<D>::threads;
    const AttnArgs &a = p.a;
    const int per = (a.batch + threads - 1) / threads;
    const int b0 = min(a.batch, static_cast<int>(threadIdx.x) * per), b1 = min(a.batch, b0 + per);
    int64_t mine = 0;
    int bad = 0;
    for (int b = b0; b < b1; ++b) {
        const RequestRows r = request_rows(a, p.page_shift, b);
        mine += request_blocks<D>(p, r);
        bad |= r.bad;
    }
    if (bad && blockIdx.x == 0) record_error(p.ctx, kDevErrIndex);
    if (threadIdx.x == 0) sh.block.b = -1;
    int64_t blocks;
    sh.blocks[threadIdx.x] = sum_before<threads>(sh, mine, blocks);
    __syncthreads();
    if (blocks > INT32_MAX / p.kv_heads) blocks = 0;  // requests that overlap: an error by now
    if (p.split == 0) {
        const int64_t at = blockIdx.x / p.kv_heads;
        if (threadIdx.x == 0 && at < blocks) {
            Walk<D> w;
            w.start(p, sh, at);
            sh.block = w.block(p, blockIdx.x - static_cast<int>(at) * p.kv_heads);
        }
        __syncthreads();
        return;
    }
    const int64_t each = (blocks + threads - 1) / threads;
    const int64_t i0 = min(blocks, threadIdx.x * each), i1 = min(blocks, i0 + each);
    Walk<D> first;
    int64_t tiles = 0, total;
    if (i0 < i1) {
        first.start(p, sh, i0);
        Walk<D> w = first;
        for (int64_t i = i0; i < i1; ++i, w.next(p)) tiles += static_cast<int64_t>(w.block(p, 0).tiles) * p.kv_heads;
    }
    sum_before<threads>(sh, tiles, total);
    const int64_t all = blocks * p.kv_heads;
    const int64_t shares = 4 * all <= 3 * p.split ? p.split - all : p.split / 2;
    const int64_t most = max(static_cast<int64_t>(kMinPart), (total + shares - 1) / shares);
    auto parts_of = [&](int n) { return n > most ? static_cast<int>((n + most - 1) / most) : 1; };
    // CTAs, and in the upper half those that have parts
    int64_t count = 0;
    if (i0 < i1) {
        Walk<D> w = first;
        for (int64_t i = i0; i < i1; ++i, w.next(p)) {
            const int n = parts_of(w.block(p, 0).tiles);
            count += (n > 1 ? (static_cast<int64_t>(n) << 32) + n : 1) * p.kv_heads;
        }
    }
    int64_t ctas;
    int64_t before = sum_before<threads>(sh, count, ctas);
    // Rows that requests claim twice can make the plan larger than the grid,
    // which is sized by total_q: parts that no CTA writes must not be joined.
    const bool fits = static_cast<uint32_t>(ctas) <= gridDim.x;
    if (threadIdx.x == 0 && blockIdx.x == 0) {
        p.header->used = fits ? static_cast<int>(ctas >> 32) : 0;
        if (!fits) record_error(p.ctx, kDevErrIndex);
    }
    if (fits && i0 < i1 && blockIdx.x >= static_cast<uint32_t>(before) && blockIdx.x < static_cast<uint32_t>(before + count)) {
        Walk<D> w = first;
        for (int64_t i = i0; i < i1; ++i, w.next(p)) {
            Block k = w.block(p, 0);
            const int n = parts_of(k.tiles);
            const int64_t here = (n > 1 ? (static_cast<int64_t>(n) << 32) + n : 1) * p.kv_heads;
            if (blockIdx.x >= static_cast<uint32_t>(before + here)) {
                before += here;
                continue;
            }
            const int at = static_cast<int>(blockIdx.x - static_cast<uint32_t>(before));
            k.kv_head = at / n;
            if (n > 1) {
                k.slot = static_cast<int>(before >> 32) + at;
                const int part = at - k.kv_head * n;
                p.parts[k.slot] = TileParts{part == 0 ? n : 0, k};
                const int t0 = static_cast<int>(static_cast<int64_t>(k.tiles) * part / n);
                const int t1 = static_cast<int>(static_cast<int64_t>(k.tiles) * (part + 1) / n);
                k.key0 += t0 * kKeys;
                k.tiles = t1 - t0;
            }
            sh.block = k;
            break;
        }
    }
    __syncthreads();
}

// ---- passes --------------------------------------------------------------------------

// All threads meet at the end of a pass and learn whether another follows.
// What they go by is written before the barrier only, so that all go the same
// way whatever happens to a wait.  Tiles are counted on through the passes,
// which keeps the phases of the barriers and the ring in step.
template <int D>
__device__ __forceinline__ bool another_pass(const TileShared &sh, int pass) {
    tc_fence_before();
    asm volatile("bar.sync 1, %0;" ::"n"(Tile<D>::threads) : "memory");
    tc_fence_after();
    return pass + 1 < kPasses && sh.again[pass] != 0;
}

// ---- dequantisation ----------------------------------------------------------------

// The 16 bytes of one block to 32 binary16 values in the words' own order, as
// four 16-byte chunks; d below 2.
// near: (n - 8) d 2^-kNear.  A code masked in place is the subnormal number
// n 2^-24 (16 n 2^-24 for the upper codes), and one multiply-add with exact
// constants gives the value, rounded once.
__device__ __forceinline__ void dequant_near(const uint4 &codes, float d, uint4 (&out)[4]) {
    const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
    const uint32_t low = pack_rn(d * 16384.0f, d * 16384.0f), high = pack_rn(d * 1024.0f, d * 1024.0f);
    const uint32_t minus = pack_rn(d * -0.0078125f, d * -0.0078125f);  // -8 2^-10
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t x = w[i], x8 = x >> 8;
        out[i].x = hfma2(x & 0x000F000Fu, low, minus);
        out[i].y = hfma2(x & 0x00F000F0u, high, minus);
        out[i].z = hfma2(x8 & 0x000F000Fu, low, minus);
        out[i].w = hfma2(x8 & 0x00F000F0u, high, minus);
    }
}
// far: (n - 8) d, by way of 1024 + n, where the scales of a tile lie so far
// apart that the smallest would leave near's values among the subnormals.
__device__ __forceinline__ void dequant_far(const uint4 &codes, float d, uint4 (&out)[4]) {
    const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
    const uint32_t magic = 0x64006400u, minus = 0xE408E408u;        // 1024, -1032
    const uint32_t sixteenth = 0x2C002C00u, minus72 = 0xD480D480u;  // 1/16, -72
    const uint32_t d2 = pack_rn(d, d);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t x = w[i], x8 = x >> 8;
        out[i].x = hmul2(hadd2((x & 0x000F000Fu) | magic, minus), d2);
        out[i].y = hmul2(hfma2((x & 0x00F000F0u) | magic, sixteenth, minus72), d2);
        out[i].z = hmul2(hadd2((x8 & 0x000F000Fu) | magic, minus), d2);
        out[i].w = hmul2(hfma2((x8 & 0x00F000F0u) | magic, sixteenth, minus72), d2);
    }
}
constexpr int kNear = 10, kNearSpan = 6;  // near: exponents of a tile's scales at most so far apart

// What a dequant thread holds of one tile: its key's blocks.
template <int D>
struct Codes {
    uint4 of[2][Tile<D>::units];
};
template <int D>
struct Scales {
    uint16_t of[2][Tile<D>::units];
    int64_t row;   // of the cache
    bool there, lost;  // the key has a page; or should have
};

template <int D>
__device__ __forceinline__ void dequant_role(const TileParams &p, TileShared &sh, uint8_t *smem, int w8, int lane) {
    using T = Tile<D>;
    constexpr int NB = D / 32, U = T::units;
    const Block bk = sh.block;
    // the thread's key in each tile, and its first block; head_dim 64: four
    // warps for K and four for V
    const int key = D == 64 ? (w8 & 3) * 16 + (lane & 15) : w8 * 8 + (lane & 7);
    const int block = D == 64 ? lane >> 4 : lane >> 3;
    const int half0 = D == 64 ? w8 >> 2 : 0, half1 = D == 64 ? half0 + 1 : 2;
    const int32_t *table = p.a.table + bk.b * p.a.table_width;
    // the page is not looked at before it is needed, which would wait for the load
    auto page_of = [&](int t) -> int32_t {
        const int k = bk.key0 + t * kKeys + key;
        if (t >= bk.tiles || k < bk.lo || k >= bk.hi) return -1;  // no key
        return table[k >> p.page_shift];
    };
    auto load_scales = [&](int t, int32_t page, Scales<D> &h) {
        const int k = bk.key0 + t * kKeys + key;
        h.there = page >= 0 && page < p.num_pages;
        h.lost = !h.there && t < bk.tiles && k >= bk.lo && k < bk.hi;
        h.row = h.there ? (((page * p.kv_heads) + bk.kv_head) << p.page_shift) + (k & ((1 << p.page_shift) - 1)) : 0;
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                h.of[half][u] = 0;
                if (h.there && half >= half0 && half < half1)
                    h.of[half][u] = reinterpret_cast<const uint16_t *>(half ? p.v_scales : p.k_scales)[h.row * NB + block + 4 * u];
            }
    };
    auto load_codes = [&](const Scales<D> &h, Codes<D> &c) {
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                c.of[half][u] = make_uint4(0u, 0u, 0u, 0u);
                if (h.there && half >= half0 && half < half1)
                    c.of[half][u] = reinterpret_cast<const uint4 *>((half ? p.v_codes : p.k_codes) + h.row * (D / 2))[block + 4 * u];
            }
    };
    int stage = 0, t = 0;
    uint32_t phase = 0;
    for (int pass = 0;; ++pass) {
        // codes a tile ahead, scales two, pages three
        int32_t page = page_of(2);
        Scales<D> scales, scales1, scales2;
        Codes<D> next;
        load_scales(0, page_of(0), scales1);
        load_scales(1, page_of(1), scales2);
        load_codes(scales1, next);
        for (int i = 0; i < bk.tiles; ++i, ++t) {
            const Codes<D> cur = next;
            scales = scales1;
            scales1 = scales2;
            load_codes(scales1, next);
            load_scales(i + 2, page, scales2);
            page = page_of(i + 3);
            // the warp's keys have one power of two for K and one for V, from the
            // largest and smallest scale: bits of binary16 order as the numbers do
            TileInfo &info = sh.info[t % kRing];
            int e[2];
            bool near[2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t top = 0, low = 0x7FFF;  // low: of those that are not 0
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    uint32_t bits = scales.of[half][u] & 0x7FFFu;
                    if (bits >= 0x7C00u) {
                        if (half && scales.there) sh.odd = 1;
                        bits = 0;  // NaN and infinity do not set the scale
                    }
                    top = max(top, bits);
                    low = min(low, bits ? bits : 0x7FFFu);
                }
                top = __reduce_max_sync(0xFFFFFFFFu, top);
                low = __reduce_min_sync(0xFFFFFFFFu, low);
                auto scale_of = [](uint32_t bits) { return exponent(__half2float(__ushort_as_half(static_cast<unsigned short>(bits)))); };
                e[half] = top ? scale_of(top) : -24;
                near[half] = !top || e[half] - scale_of(low) <= kNearSpan;
            }
            if (__any_sync(0xFFFFFFFFu, scales.lost) && lane == 0) {
                record_error(p.ctx, kDevErrIndex);
                atomicOr(&info.lost, 1u << (key >> 4));  // lane 0's key: the warp's keys lie in one group
            }
            if (lane == 0) {
                const float k_unit = pow2i(e[0] + (near[0] ? kNear : 0));
                const int v_exp = near[1] ? 2 * (e[1] + kNear) : 2 * e[1] + 1;
                if constexpr (D == 64) {
                    if (half0 == 0)
                        info.k_unit[2 * w8] = info.k_unit[2 * w8 + 1] = k_unit;
                    else
                        info.v_exp[2 * w8 - 8] = info.v_exp[2 * w8 - 7] = v_exp;
                } else {
                    info.k_unit[w8] = k_unit;
                    info.v_exp[w8] = v_exp;
                }
                if (w8 == 0)  // not in use: the warps' and the readers' tiles lie less apart
                    sh.info[(t + kRing / 2) % kRing].lost = 0;
            }
            if (!warp_wait_or_abort(smem_addr(sh.k_empty + stage), phase ^ 1u, &sh.abort, p.ctx) ||
                !warp_wait_or_abort(smem_addr(sh.v_empty + stage), phase ^ 1u, &sh.abort, p.ctx))
                break;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (half < half0 || half >= half1) continue;
                uint8_t *rows = smem + (half * T::stages + stage) * T::bytes + key * 128;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int b = block + 4 * u;
                    float d = __half2float(__ushort_as_half(scales.of[half][u]));
                    if (half && !(fabsf(d) <= 65504.0f)) d = 0.0f;  // marked in sh.odd: rows that do not see the key must not either
                    d *= pow2i(-e[half]);
                    uint4 out[4];
                    if (near[half])
                        dequant_near(cur.of[half][u], d, out);
                    else
                        dequant_far(cur.of[half][u], d, out);
                    uint8_t *panel = rows + (b >> 1) * kPanel;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        *reinterpret_cast<uint4 *>(panel + ((((b & 1) * 4 + i) ^ (key & 7)) << 4)) = out[i];
                }
            }
            fence_proxy_async_smem();  // generic writes -> tensor-core reads
            __syncwarp();
            if (lane == 0) {
                mbar_arrive_addr(smem_addr(sh.k_full + stage));
                mbar_arrive_addr(smem_addr(sh.v_full + stage));
            }
            if (++stage == T::stages) {
                stage = 0;
                phase ^= 1u;
            }
        }
        if (!another_pass<D>(sh, pass)) break;
    }
}

// ---- the products --------------------------------------------------------------------

// One lane of a warp, the same each time.
__device__ __forceinline__ uint32_t elected() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one;
}
// By the elected lane; the whole warp comes here with the same operands.
__device__ __forceinline__ void product(uint32_t one, uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(one)
        : "memory");
}
__device__ __forceinline__ void products_done(uint32_t one, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(one)
        : "memory");
}

// 0xFFFF in each half that is less than binary16's normal numbers, of two that
// are not negative (NaN is not less).
__device__ __forceinline__ uint32_t subnormal2(uint32_t v) {
    return __hlt2_mask(*reinterpret_cast<const __half2 *>(&v), __half2half2(__ushort_as_half(static_cast<unsigned short>(0x0400))));
}

// The whole warp, so that the operands are known to be the same for all lanes:
// a thread on its own has to move each to the uniform registers that the
// products take theirs from.
template <int D>
__device__ __forceinline__ void mma_role(const TileParams &p, TileShared &sh, uint32_t smem_in, uint32_t tmem_in, int qt) {
    using T = Tile<D>;
    const uint32_t smem = __shfl_sync(0xFFFFFFFFu, smem_in, 0), tmem = __shfl_sync(0xFFFFFFFFu, tmem_in, 0);
    const int tiles = __shfl_sync(0xFFFFFFFFu, sh.block.tiles, 0);
    constexpr int ahead = 2 / T::QT;  // S buffers of a row tile: S of so many tiles is formed ahead
    constexpr uint32_t qk_desc = tile_idesc(kKeys, false), pv_desc = tile_idesc(D, true);
    const uint32_t one = elected();
    int *abort = &sh.abort;
    bool issued = false;
    auto qk = [&](int t) -> bool {
        const int stage = t % T::stages, buf = T::buffer(t, qt);
        if (!warp_wait_or_abort(smem_addr(sh.k_full + stage), (t / T::stages) & 1u, abort, p.ctx)) return false;
        tc_fence_after();
        const uint64_t b0 = sw128_desc(smem + stage * T::bytes);
        const uint32_t to = tmem + T::s_col + buf * kKeys, from = tmem + T::q_col + qt * (D / 2);
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
            product(one, to, from + s * 8, b0 + (((s >> 2) * kPanel + (s & 3) * 32) >> 4), qk_desc, s > 0);
        issued = true;
        products_done(one, smem_addr(sh.s_full + buf));
        products_done(one, smem_addr(sh.k_empty + stage));
        return true;
    };
    bool ok = tiles == 0 || warp_wait_or_abort(smem_addr(&sh.q_ready), 0, abort, p.ctx);
    int first = 0;  // tile of the pass
    for (int pass = 0;; ++pass, first += tiles) {
        const int end = first + tiles;
        for (int t = first; ok && t < min(first + ahead, end); ++t) ok = qk(t);
        for (int t = first; ok && t < end; ++t) {
            const int stage = t % T::stages, buf = T::buffer(t, qt);
            ok = warp_wait_or_abort(smem_addr(sh.p_full + buf), T::phase(t), abort, p.ctx) &&
                 warp_wait_or_abort(smem_addr(sh.v_full + stage), (t / T::stages) & 1u, abort, p.ctx);
            if (!ok) break;
            tc_fence_after();
            const uint64_t b0 = rows_desc(smem + (T::stages + stage) * T::bytes);
            const uint32_t to = tmem + T::o_col + qt * D, from = tmem + T::s_col + buf * kKeys;
#pragma unroll
            for (int s = 0; s < kKeys / 16; ++s) product(one, to, from + s * 8, b0 + ((s * 2048) >> 4), pv_desc, t > first || s > 0);
            products_done(one, smem_addr(sh.pv_done + qt));
            products_done(one, smem_addr(sh.v_empty + stage));
            // the next S goes where P lies, once its product has read it (products
            // with different accumulators are not ordered among themselves)
            if (t + ahead < end) ok = warp_wait_or_abort(smem_addr(sh.pv_done + qt), t & 1u, abort, p.ctx) && qk(t + ahead);
        }
        if (!another_pass<D>(sh, pass)) break;
    }
    if (issued) {  // all products end before tensor memory is freed
        products_done(one, smem_addr(sh.final + qt));
        wait_drain(smem_addr(sh.final + qt), 0, p.ctx);
    }
}

// ---- softmax ----------------------------------------------------------------------------

// Eight consecutive values of a row of q.
__device__ __forceinline__ void load8(const AttnArgs &a, int64_t at, bool wide, float (&v)[8]) {
    if (wide && a.q_bf16) {
        const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) + at);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else if (wide) {
        const float4 x = *reinterpret_cast<const float4 *>(static_cast<const float *>(a.q) + at);
        const float4 y = *reinterpret_cast<const float4 *>(static_cast<const float *>(a.q) + at + 4);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = load_value(a.q, at + i, a.q_bf16);
    }
}

// Value d of a block is at this place of the order in which words give them.
__host__ __device__ constexpr int place_of(int d) {
    return ((d & 15) >> 2) * 8 + ((d & 1) << 2) + ((d >> 4) << 1) + ((d >> 1) & 1);
}

// A warp looks over the values of one block of V, for the keys of this CTA's
// tiles: in which digits of the codes some value is not 0, and whether a key of
// the lane's row (from lo up to hi) has one that is no number.  It is seldom
// asked: where the dequantisers met such a number, and where an output that
// lost weights might matter to is exactly 0.  `want`: digits in question, after
// whose last the rest is left; or none, for all keys.  The warp takes the keys'
// `part`th of every `parts` batches.
template <int D>
__device__ __noinline__ uint4 look_over(const TileParams &p, const Block &bk, int b, int lo, int hi, const uint4 &want, int part, int parts,
                                        bool &odd) {
    constexpr int kBatch = 8, NB = D / 32;
    const int step = 32 * kBatch * parts;
    const int lane = threadIdx.x & 31, from = max(bk.lo, bk.key0) + 32 * kBatch * part;
    const int to = min(bk.hi, bk.key0 + bk.tiles * kKeys);
    const int32_t *table = p.a.table + bk.b * p.a.table_width;
    uint32_t live[4] = {};
    int32_t page[kBatch];
    auto load_pages = [&](int key0) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int key = key0 + 32 * j + lane;
            page[j] = key < to ? table[key >> p.page_shift] : -1;
        }
    };
    load_pages(from);
#pragma unroll 1
    for (int key0 = from; key0 < to; key0 += step) {
        uint32_t bits[kBatch];
        uint4 codes[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int key = key0 + 32 * j + lane;
            bits[j] = 0;
            codes[j] = make_uint4(0u, 0u, 0u, 0u);
            if (page[j] >= 0 && page[j] < p.num_pages) {
                const int64_t row = (((page[j] * p.kv_heads) + bk.kv_head) << p.page_shift) + (key & ((1 << p.page_shift) - 1));
                bits[j] = reinterpret_cast<const uint16_t *>(p.v_scales)[row * NB + b] & 0x7FFFu;
                codes[j] = reinterpret_cast<const uint4 *>(p.v_codes + row * (D / 2))[b];
            }
        }
        load_pages(min(key0, to - step) + step);  // a batch ahead
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            if (bits[j]) {
                live[0] |= codes[j].x ^ 0x88888888u, live[1] |= codes[j].y ^ 0x88888888u;
                live[2] |= codes[j].z ^ 0x88888888u, live[3] |= codes[j].w ^ 0x88888888u;
            }
            for (unsigned keys = __ballot_sync(0xFFFFFFFFu, bits[j] >= 0x7C00u); keys; keys &= keys - 1u) {
                const int key = key0 + 32 * j + __ffs(keys) - 1;
                odd |= key >= lo && key < hi;
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) live[k] = __reduce_or_sync(0xFFFFFFFFu, live[k]);
        auto dead = [](uint32_t digits, uint32_t of) { return of & ~(digits | digits >> 1 | digits >> 2 | digits >> 3) & 0x11111111u; };
        const bool any = want.x | want.y | want.z | want.w;
        if (any && !(dead(live[0], want.x) | dead(live[1], want.y) | dead(live[2], want.z) | dead(live[3], want.w))) break;
    }
    return make_uint4(live[0], live[1], live[2], live[3]);
}

template <int D>
__device__ __forceinline__ void softmax_barrier() {
    asm volatile("bar.sync 2, %0;" ::"n"(Tile<D>::softmax_warps * 32) : "memory");
}

// Where value d of a block stands among the digits of its codes: word and shift.
__host__ __device__ constexpr int digit_word(int d) { return (d & 15) >> 2; }
__host__ __device__ constexpr int digit_shift(int d) { return (d & 3) * 8 + (d >> 4) * 4; }

template <int D>
__device__ __forceinline__ void softmax_role(const TileParams &p, TileShared &sh, uint32_t tmem, int warp, int lane) {
    using T = Tile<D>;
    constexpr int NB = D / 32;
    const AttnArgs &a = p.a;
    const Block bk = sh.block;
    const int qt = warp >> 2, row = warp * 32 + lane, heads = a.heads / p.kv_heads;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float ninf = __uint_as_float(0xFF800000u);
    const bool mine = row < bk.rows;
    const int flat = bk.flat0 + (mine ? row : 0), token = flat / heads, head = bk.kv_head * heads + flat - token * heads;
    const int64_t q_at = (static_cast<int64_t>(bk.q_row0) + token) * a.q_stride + static_cast<int64_t>(head) * D;

    // the row of q, scaled to below 2^15, into tensor memory
    const float size = fabsf(a.scale) * kLog2e, sign = !mine || a.scale == 0.0f ? 0.0f : a.scale < 0.0f ? -1.0f : 1.0f;
    float unit;
    if (bk.tiles > 0) {
        uint32_t bits = 0;  // of the largest value: positive numbers order as their bits do
        float f;
        const uint32_t q_to = tmem + lanes + T::q_col + qt * (D / 2);
        auto scale_up = [&]() {
            const int up = query_raise(sign == 0.0f ? 0.0f : __uint_as_float(bits), size);
            f = pow2i(up) * sign;
            unit = score_unit(size, -up);
        };
        if (a.q_bf16 && p.q_wide) {  // 128 values of a row under way at once; the last are kept for the second pass
            constexpr int C = D / 8 < 16 ? D / 8 : 16, H = D / 8 / C;
            uint4 raw[C];
            const uint4 *from = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) + q_at);
            auto load = [&](int h) {
#pragma unroll
                for (int i = 0; i < C; ++i) raw[i] = from[h * C + i];
            };
#pragma unroll 1
            for (int h = H - 1; h >= 0; --h) {
                load(h);
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) bits = max(bits, max((w[k] & 0x7FFFu) << 16, w[k] & 0x7FFF0000u));
                }
            }
            scale_up();
#pragma unroll 1
            for (int h = 0; h < H; ++h) {
                if (h > 0) load(h);
#pragma unroll
                for (int b = 0; b < C / 4; ++b) {
                    uint32_t cols[16];
                    auto value = [&](int d) {
                        const uint4 &r = raw[b * 4 + (d >> 3)];
                        const uint32_t w = (d >> 1 & 3) == 0 ? r.x : (d >> 1 & 3) == 1 ? r.y : (d >> 1 & 3) == 2 ? r.z : r.w;
                        return __uint_as_float(d & 1 ? w & 0xFFFF0000u : w << 16) * f;
                    };
#pragma unroll
                    for (int i = 0; i < 16; ++i) {  // values d and d + 2 stand side by side
                        const int d = ((i >> 2) << 2) + ((i >> 1) & 1) + ((i & 1) << 4);
                        cols[i] = pack_rn(value(d), value(d + 2));
                    }
                    tmem_st_16cols(q_to + (h * (C / 4) + b) * 16, cols);
                }
            }
        } else {
#pragma unroll 1
            for (int i = 0; i < D; i += 64) {
                float v[8][8];
#pragma unroll
                for (int c = 0; c < 8; ++c) load8(a, q_at + i + c * 8, p.q_wide, v[c]);
#pragma unroll
                for (int c = 0; c < 8; ++c)
#pragma unroll
                    for (int k = 0; k < 8; ++k) bits = max(bits, __float_as_uint(v[c][k]) & 0x7FFFFFFFu);
            }
            scale_up();
#pragma unroll 1
            for (int b = 0; b < NB; b += 2) {
                float v[2][32];
#pragma unroll
                for (int i = 0; i < 64; i += 8) {
                    float u[8];
                    load8(a, q_at + b * 32 + i, p.q_wide, u);
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[i >> 5][(i & 31) + k] = u[k];
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t cols[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int d = ((i >> 2) << 2) + ((i >> 1) & 1) + ((i & 1) << 4);
                        cols[i] = pack_rn(v[h][d] * f, v[h][d + 2] * f);
                    }
                    tmem_st_16cols(q_to + (b + h) * 16, cols);
                }
            }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_addr(smem_addr(&sh.q_ready));
    }

    const int pos = bk.first + token;
    const int lo = mine ? first_key(a, pos) : 0, hi = mine ? (a.causal ? min(bk.len, pos + 1) : bk.len) : 0;
    float total = 0.0f; // of the weights
    uint32_t odd = 0;   // blocks of the output that a seen value leaves without a number, a bit each
    bool far = false;   // a tile was far
    bool ok = true, open = mine;  // open: what was lost of the weights may show in the row
    int first = 0;      // tile of the pass
    for (int pass = 0;; ++pass, first += bk.tiles) {
        float top = ninf;   // the weights' reference (2^kRaise there)
        int e_ref = -24;    // exponent of V's unit in O
        float sum = 0.0f;   // of the weights (first pass)
        int faint = 0;      // tiles in which a weight fell below binary16's normal numbers
        auto tiles = [&](auto is_later) {
            constexpr bool later = decltype(is_later)::value;
            for (int t = first; ok && t < first + bk.tiles; ++t) {
                const int buf = T::buffer(t, qt);
                if (!warp_wait_or_abort(smem_addr(sh.s_full + buf), T::phase(t), &sh.abort, p.ctx) ||
                    !warp_wait_or_abort(smem_addr(sh.v_full + t % T::stages), (t / T::stages) & 1u, &sh.abort, p.ctx)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (later && !__any_sync(0xFFFFFFFFu, open)) {  // nothing of these rows is wanted: any weights do
                    if (t > 0 && !warp_wait_or_abort(smem_addr(sh.pv_done + qt), (t - 1) & 1u, &sh.abort, p.ctx)) {
                        ok = false;
                        break;
                    }
                    tc_fence_before();
                    if (lane == 0) mbar_arrive_addr(smem_addr(sh.p_full + buf));
                    continue;
                }
                const uint32_t s_at = tmem + lanes + T::s_col + buf * kKeys;
                uint32_t s[64];
                tmem_ld_64cols(s_at, s);
                const TileInfo &info = sh.info[t % kRing];
                float u[8];
                int v_exp[8], most_exp = -0x10000;
#pragma unroll
                for (int g = 0; g < 8; g += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(info.k_unit + g);
                    const int4 e = *reinterpret_cast<const int4 *>(info.v_exp + g);
                    u[g] = unit * f.x, u[g + 1] = unit * f.y, u[g + 2] = unit * f.z, u[g + 3] = unit * f.w;
                    far |= (e.x | e.y | e.z | e.w) & 1;
                    v_exp[g] = e.x >> 1, v_exp[g + 1] = e.y >> 1, v_exp[g + 2] = e.z >> 1, v_exp[g + 3] = e.w >> 1;
                    most_exp = max(max(most_exp, max(v_exp[g], v_exp[g + 1])), max(v_exp[g + 2], v_exp[g + 3]));
                }
                const int key0 = bk.key0 + (t - first) * kKeys;
                const bool edge = info.lost || key0 < bk.lo_all || key0 + kKeys > bk.hi_all;
                if (edge) {
                    const uint32_t lost = info.lost;
#pragma unroll
                    for (int i = 0; i < 64; ++i)
                        if (key0 + i < lo || key0 + i >= hi || ((lost >> (i >> 4)) & 1u)) s[i] = 0xFF800000u;
                }
                float here = ninf;
#pragma unroll
                for (int g = 0; g < 8; ++g) {
                    float most = __uint_as_float(s[8 * g]);
#pragma unroll
                    for (int k = 1; k < 7; k += 2) most = fmaxf(most, fmaxf(__uint_as_float(s[8 * g + k]), __uint_as_float(s[8 * g + k + 1])));
                    here = fmaxf(here, fmaxf(most, __uint_as_float(s[8 * g + 7])) * u[g]);
                }
                // a new reference where the largest weight would pass 2^15, and where
                // V's unit grows
                const bool grow = here > top + kSlack;
                const int e_now = max(e_ref, most_exp);
                const float now = grow || top == ninf ? fmaxf(top, here) : top;
                if (__any_sync(0xFFFFFFFFu, now != top || e_now != e_ref)) {
                    const float f = top == ninf ? 0.0f : exp2_fast(top - now);
                    sum *= f;
                    if (t > first) {
                        const float scale = f * pow2i(e_ref - e_now);
                        if (!warp_wait_or_abort(smem_addr(sh.pv_done + qt), (t - 1) & 1u, &sh.abort, p.ctx)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            uint32_t o[32], v[16];
                            const uint32_t at = tmem + lanes + T::o_col + qt * D + c;
                            tmem_ld_32cols(at, o);
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
#pragma unroll
                                for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(o[16 * h + i]) * scale);
                                tmem_st_16cols(at + 16 * h, v);
                            }
                        }
                    }
                    top = now;
                    e_ref = e_now;
                }
                const float top_here = top == ninf ? 0.0f : top;
                float base[8];
#pragma unroll
                for (int g = 0; g < 8; ++g)
                    base[g] = static_cast<float>(kRaise + (later ? kPassRaise * (pass - 1) : 0) + v_exp[g] - e_ref) - top_here;
                if constexpr (later) {
                    // What the pass before has lost of the weights.  z, a weight as
                    // that pass had it (within 2^-16 of it, far less than what this one
                    // adds), is a subnormal number there or 0; weights that were so
                    // one pass earlier still leave nothing to it.
                    const float raise = pow2i(kPassRaise);
                    bool low = false;
                    if (edge) {
#pragma unroll
                        for (int i = 0; i < 64; ++i)
                            low |= s[i] != 0xFF800000u && fmaf(__uint_as_float(s[i]), u[i >> 3], base[i >> 3]) <
                                                              static_cast<float>(-14 - kPassRaise);
                    }
                    float smallest = 1.0f;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t w[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int g = 4 * h + (i >> 2);
                            const float2 arg = __ffma2_rn(make_float2(__uint_as_float(s[32 * h + 2 * i]), __uint_as_float(s[32 * h + 2 * i + 1])),
                                                          make_float2(u[g], u[g]), make_float2(base[g], base[g]));
                            const float2 z = make_float2(exp2_fast(arg.x), exp2_fast(arg.y));
                            const uint32_t had = pack_rn(z.x, z.y);
                            const float2 lost = __fadd2_rn(z, make_float2(-low_float(had), -high_float(had)));
                            const float2 y = __fmul2_rn(lost, make_float2(raise, raise));
                            w[i] = pack_rn(y.x, y.y) & subnormal2(had);
                            smallest = fminf(smallest, fminf(z.x, z.y));
                        }
                        tmem_st_16cols(s_at + 16 * h, w);
                    }
                    if (!edge) low = smallest * raise < kNormal;
                    faint += low ? 1 : 0;
                } else {
                    bool low = false;
                    if (edge) {  // hidden keys' weights are 0 and do not count
#pragma unroll
                        for (int i = 0; i < 64; ++i)
                            low |= s[i] != 0xFF800000u && fmaf(__uint_as_float(s[i]), u[i >> 3], base[i >> 3]) < -14.0f;
                    }
                    uint32_t least[2] = {0x7C007C00u, 0x7C007C00u};  // smallest weights
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t w[16];
#pragma unroll
                        for (int g = 4 * h; g < 4 * h + 4; ++g) {
                            float2 add = make_float2(0.0f, 0.0f);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float2 arg = __ffma2_rn(make_float2(__uint_as_float(s[8 * g + 2 * i]), __uint_as_float(s[8 * g + 2 * i + 1])),
                                                              make_float2(u[g], u[g]), make_float2(base[g], base[g]));
                                const float2 x = make_float2(exp2_fast(arg.x), exp2_fast(arg.y));
                                add = i == 0 ? x : __fadd2_rn(add, x);
                                const uint32_t both = pack_rn(x.x, x.y);
                                w[4 * (g & 3) + i] = both;
                                least[i & 1] = hmin2(least[i & 1], both);
                            }
                            sum = fmaf(add.x + add.y, pow2i(e_ref - kRaise - v_exp[g]), sum);
                        }
                        tmem_st_16cols(s_at + 16 * h, w);
                    }
                    least[0] = hmin2(least[0], least[1]);
                    if (!edge) low = (least[0] & 0x7C00u) == 0 || (least[0] & 0x7C000000u) == 0;  // below the normal numbers
                    faint += low ? 1 : 0;
                }
                // Every phase of pv_done is waited for in turn, before the next product
                // can start: a barrier's parity tells neighbouring phases apart only.
                if (t > 0 && !warp_wait_or_abort(smem_addr(sh.pv_done + qt), (t - 1) & 1u, &sh.abort, p.ctx)) {
                    ok = false;
                    break;
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_addr(smem_addr(sh.p_full + buf));
            }
        };
        // Code of its own spares the first pass the test, which costs 5 us of 195
        // (2048 tokens behind 6000) and of 99 (the windowed prompts).
        if (pass == 0)
            tiles(std::false_type{});
        else
            tiles(std::true_type{});
        if (pass == 0) total = sum;

        // outputs
        if (ok && bk.tiles > 0) ok = warp_wait_or_abort(smem_addr(sh.pv_done + qt), (first + bk.tiles - 1) & 1u, &sh.abort, p.ctx);
        tc_fence_after();
        // A faint weight is off by at most 2^-25, times values below 16 (near tiles
        // only: 2^-6), a key.  Scores that lie 24 powers of two apart are
        // themselves uncertain by more than 2^-6 of a weight (binary16 q and K,
        // A >= 8), so an output has to be 2^6 times that sum at least.
        const float error = static_cast<float>(faint * kKeys) * (far ? pow2i(-15) : pow2i(-15 - kNear));
        const float back = pow2i(e_ref - kRaise);  // of O's unit
        const float down = bk.slot >= 0 ? back : total == 0.0f ? 0.0f : back / total;
        const float raised = pow2i(-kPassRaise * pass);
        if (sh.odd && pass == 0) {
#pragma unroll 1
            for (int b = 0; b < NB; ++b) {
                bool here = false;
                look_over<D>(p, sh.block, b, lo, hi, make_uint4(0u, 0u, 0u, 0u), 0, 1, here);
                if (here) odd |= 1u << b;
            }
        }
        // the row's smallest output, in units of `down` (or, where outputs are
        // added to, as it is)
        float least = __uint_as_float(0x7F800000u);
        auto live_of = [&](int b) {
            const uint4 z = *reinterpret_cast<const uint4 *>(sh.zero[b]), f = *reinterpret_cast<const uint4 *>(sh.found[b]);
            return make_uint4(f.x | ~z.x, f.y | ~z.y, f.z | ~z.z, f.w | ~z.w);
        };
        auto look_at = [&](const uint4 &live4, int d, float v) {  // of the outputs that some value enters
            const int k = digit_word(d);
            const uint32_t live = k == 0 ? live4.x : k == 1 ? live4.y : k == 2 ? live4.z : live4.w;
            if (live & (15u << digit_shift(d))) least = fminf(least, fabsf(v));
        };
        if (ok) {
            const int64_t out_row = static_cast<int64_t>(bk.q_row0) + token;
            const int64_t out_at = out_row * a.out_stride + static_cast<int64_t>(head) * D;
            float *rec = p.records + static_cast<int64_t>(max(bk.slot, 0)) * kPartFloats;  // the joining kernel goes on
            float4 *rec_to = reinterpret_cast<float4 *>(rec) + (row >> 3) * (D / 4 * 8) + (row & 7);
#pragma unroll 1
            for (int b = 0; b < NB; ++b) {
                uint32_t o[32];
                __syncwarp();  // rows that have nothing to write went ahead
                if (bk.tiles > 0) {
                    tmem_ld_32cols(tmem + lanes + T::o_col + qt * D + b * 32, o);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0u;
                }
                const float unit_out = (odd >> b) & 1u ? __uint_as_float(0x7FFFFFFFu) : down;
                if (__builtin_expect(pass > 0, 0)) {
                    // added to what this thread wrote before, and rounded once more
                    // (within what the row's scores leave uncertain)
                    if (!open) continue;
                    const float raised_out = raised * unit_out;
                    const uint4 live4 = live_of(b);
                    auto add = [&](int d, float had) {
                        const float v = fmaf(__uint_as_float(o[place_of(d)]), raised_out, had);
                        look_at(live4, d, v);
                        return v;
                    };
                    if (bk.slot >= 0) {
#pragma unroll
                        for (int d = 0; d < 32; d += 4) {
                            float4 &to = rec_to[(b * 8 + d / 4) * 8];
                            to = make_float4(add(d, to.x), add(d + 1, to.y), add(d + 2, to.z), add(d + 3, to.w));
                        }
                    } else if (p.out_wide) {
                        uint4 *to = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + out_at + b * 32);
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const uint4 had = to[c];
                            uint32_t w[4] = {had.x, had.y, had.z, had.w};
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int d = c * 8 + i * 2;
                                w[i] = pack_bf16x2(add(d, __uint_as_float(w[i] << 16)), add(d + 1, __uint_as_float(w[i] & 0xFFFF0000u)));
                            }
                            to[c] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    } else {
#pragma unroll
                        for (int d = 0; d < 32; ++d)
                            store_value(a.out, out_at + b * 32 + d, true, add(d, load_value(a.out, out_at + b * 32 + d, true)));
                    }
                    continue;
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) least = fminf(least, fabsf(__uint_as_float(o[i])));
                if (!mine) continue;
                if (bk.slot >= 0) {
#pragma unroll
                    for (int d = 0; d < 32; d += 4)
                        rec_to[(b * 8 + d / 4) * 8] = make_float4(
                            __uint_as_float(o[place_of(d)]) * unit_out, __uint_as_float(o[place_of(d + 1)]) * unit_out,
                            __uint_as_float(o[place_of(d + 2)]) * unit_out, __uint_as_float(o[place_of(d + 3)]) * unit_out);
                } else if (p.out_wide) {
                    uint4 *to = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + out_at + b * 32);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int d = c * 8 + i * 2;
                            w[i] = pack_bf16x2(__uint_as_float(o[place_of(d)]) * unit_out, __uint_as_float(o[place_of(d + 1)]) * unit_out);
                        }
                        to[c] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                } else {
#pragma unroll
                    for (int d = 0; d < 32; ++d)
                        store_value(a.out, out_at + b * 32 + d, true, __uint_as_float(o[place_of(d)]) * unit_out);
                }
            }
            if (pass == 0 && mine) {
                if (bk.slot >= 0)
                    *reinterpret_cast<float2 *>(rec + T::rows * D + row * 2) = make_float2(top, total);
                else if (a.lse)
                    a.lse[out_row * a.heads + head] = total == 0.0f ? ninf : (top + log2f(total)) * kLn2;
            }
        }
        open = open && ok && least < (pass == 0 ? error : error * raised * down);
        if (pass == 0) {  // outputs of exactly 0 in which every value is 0 do not count
            const bool any_open = __any_sync(0xFFFFFFFFu, open);
            if (any_open) {
#pragma unroll 1
                for (int b = 0; b < NB; ++b) {
                    uint32_t o[32], zero[4] = {};
                    tmem_ld_32cols(tmem + lanes + T::o_col + qt * D + b * 32, o);
#pragma unroll
                    for (int d = 0; d < 32; ++d)
                        if (__uint_as_float(o[place_of(d)]) == 0.0f) zero[digit_word(d)] |= 15u << digit_shift(d);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        zero[k] = __reduce_and_sync(0xFFFFFFFFu, open ? zero[k] : ~0u);  // in all such rows
                        if (lane == 0 && zero[k]) {
                            atomicOr(&sh.zero[b][k], zero[k]);
                            sh.any_zero = 1;
                        }
                    }
                }
            }
            softmax_barrier<D>();
            if (sh.any_zero) {
#pragma unroll 1
                for (int b = 0; b < NB; ++b) {
                    const uint4 want = *reinterpret_cast<const uint4 *>(sh.zero[b]);
                    if (!(want.x | want.y | want.z | want.w)) continue;
                    bool unused = false;
                    const uint4 f = look_over<D>(p, sh.block, b, lo, hi, want, warp, T::softmax_warps, unused);
                    if (lane < 4) atomicOr(&sh.found[b][lane], lane == 0 ? f.x : lane == 1 ? f.y : lane == 2 ? f.z : f.w);
                }
                softmax_barrier<D>();
                if (any_open) {
                    least = __uint_as_float(0x7F800000u);
#pragma unroll 1
                    for (int b = 0; b < NB; ++b) {
                        uint32_t o[32];
                        tmem_ld_32cols(tmem + lanes + T::o_col + qt * D + b * 32, o);
                        const uint4 live4 = live_of(b);
#pragma unroll
                        for (int d = 0; d < 32; ++d) look_at(live4, d, __uint_as_float(o[place_of(d)]));
                    }
                    open = open && least < error;
                }
            }
        }
        if (__any_sync(0xFFFFFFFFu, open) && lane == 0) sh.again[pass] = 1;
        if (!another_pass<D>(sh, pass)) break;
    }
}

template <int D>
__global__ void __launch_bounds__(Tile<D>::threads, 1) attn_tile_kernel(const __grid_constant__ TileParams p) {
    using T = Tile<D>;
    extern __shared__ uint8_t tile_smem[];
    uint8_t *smem = tile_smem + ((1024u - (smem_addr(tile_smem) & 1023u)) & 1023u);
    TileShared &sh = *reinterpret_cast<TileShared *>(smem + 2 * T::stages * T::bytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == T::mma_warp * 32) {
        for (int i = 0; i < T::stages; ++i) {
            mbar_init(sh.k_full + i, kDequantWarps);
            mbar_init(sh.k_empty + i, T::QT);
            mbar_init(sh.v_full + i, kDequantWarps);
            mbar_init(sh.v_empty + i, T::QT);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(sh.s_full + i, 1);
            mbar_init(sh.p_full + i, 4);
            mbar_init(sh.pv_done + i, 1);
            mbar_init(sh.final + i, 1);
        }
        mbar_init(&sh.q_ready, T::softmax_warps);
        sh.abort = 0;
        fence_mbar_init();
    }
    for (int i = threadIdx.x; i < kRing; i += T::threads) sh.info[i] = TileInfo{};
    if (threadIdx.x < kPasses) sh.again[threadIdx.x] = 0;
    if (threadIdx.x == 0) sh.odd = sh.any_zero = 0;
    if (threadIdx.x < 32) sh.zero[threadIdx.x >> 2][threadIdx.x & 3] = sh.found[threadIdx.x >> 2][threadIdx.x & 3] = 0;
    pdl_wait();
    pdl_launch_dependents();
    find_block<D>(p, sh);
    if (sh.block.b < 0) return;  // the whole CTA
    if (warp == T::mma_warp) tmem_alloc_cta(smem_addr(&sh.tmem), T::tmem_cols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(&sh.tmem);

    if (warp < T::softmax_warps) {
        registers_up<T::softmax_regs>();
        softmax_role<D>(p, sh, tmem, warp, lane);
    } else if (warp < T::mma_warp) {
        registers_down<T::dequant_regs>();
        dequant_role<D>(p, sh, smem, warp - T::softmax_warps, lane);
    } else {
        registers_down<T::mma_regs>();
        if (warp < T::mma_warp + T::QT) {
            mma_role<D>(p, sh, smem_addr(smem), tmem, warp - T::mma_warp);
        } else {
            for (int pass = 0; another_pass<D>(sh, pass);) ++pass;
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == T::mma_warp) tmem_dealloc_cta(tmem, T::tmem_cols);
}

// Joins the parts of split blocks, eight rows at a time: a lane has four
// values of each of Q quads of one row.  Bound by the latency of its loads,
// which come from L2.
template <int D>
struct Join {
    static constexpr int warps = D == 64 ? 4 : 8, Q = D / 16 / warps, slices = Tile<D>::rows / 8;
};

template <int D>
__global__ void __launch_bounds__(Join<D>::warps * 32) attn_tile_join_kernel(const __grid_constant__ TileParams p) {
    using T = Tile<D>;
    using J = Join<D>;
    constexpr int W = J::warps, Q = J::Q;
    __shared__ int starts[kMaxTileCtas], counts[kMaxTileCtas];
    __shared__ int chains;
    __shared__ float weight[kMaxTileCtas][8];
    __shared__ float red[W][8];
    pdl_wait();
    pdl_launch_dependents();
    const AttnArgs &a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float ninf = __uint_as_float(0xFF800000u);
    const int used = p.header->used;
    if (used == 0) return;
    if (warp == 0) {
        int k = 0;
        for (int i = 0; i < used; i += 32) {
            const int n = i + lane < used ? p.parts[i + lane].count : 0;
            const unsigned have = __ballot_sync(0xFFFFFFFFu, n > 0);
            if (n > 0) {
                const int at = k + __popc(have & ((1u << lane) - 1u));
                starts[at] = i + lane;
                counts[at] = n;
            }
            k += __popc(have);
        }
        if (lane == 0) chains = k;
    }
    __syncthreads();
#pragma unroll 1
    for (int item = blockIdx.x; item < chains * J::slices; item += gridDim.x) {
        const int c = starts[item / J::slices], k = counts[item / J::slices], row0 = item % J::slices * 8;
        const Block &block = p.parts[c].block;
        if (row0 >= block.rows) continue;
        const int row = row0 + (lane & 7);
        const bool mine = row < block.rows;
        auto record = [&](int i) { return p.records + static_cast<int64_t>(c + i) * kPartFloats; };
        // the parts' weights: thread (lane & 7) of parts i, i + 4 W, ...
        const int i0 = threadIdx.x >> 3;
        float top = ninf;
        for (int i = i0; i < k; i += W * 4) {
            const float t = mine ? record(i)[T::rows * D + row * 2] : ninf;
            weight[i][lane & 7] = t;
            top = fmaxf(top, t);
        }
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 8));
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 16));
        if (lane < 8) red[warp][lane] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < W; ++w) top = fmaxf(top, red[w][lane & 7]);
        __syncthreads();
        const float ref = top == ninf ? 0.0f : top;
        float sum = 0.0f;
        for (int i = i0; i < k; i += W * 4) {
            const float2 s = mine ? *reinterpret_cast<const float2 *>(record(i) + T::rows * D + row * 2) : make_float2(ninf, 0.0f);
            const float f = exp2_fast(s.x - ref);
            weight[i][lane & 7] = f;
            sum = fmaf(f, s.y, sum);
        }
#pragma unroll
        for (int o = 8; o < 32; o <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if (lane < 8) red[warp][lane] = sum;
        __syncthreads();
        sum = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) sum += red[w][lane & 7];
        float4 v[Q];
#pragma unroll
        for (int q = 0; q < Q; ++q) v[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (mine) {
#pragma unroll 4
            for (int i = 0; i < k; ++i) {
                const float4 *from = reinterpret_cast<const float4 *>(record(i)) + (row0 >> 3) * (D / 4 * 8) + warp * Q * 32 + lane;
                const float f = weight[i][lane & 7];
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    const float4 x = from[q * 32];
                    v[q].x = fmaf(f, x.x, v[q].x);
                    v[q].y = fmaf(f, x.y, v[q].y);
                    v[q].z = fmaf(f, x.z, v[q].z);
                    v[q].w = fmaf(f, x.w, v[q].w);
                }
            }
        }
        const int heads = a.heads / p.kv_heads, flat = block.flat0 + (mine ? row : 0), token = flat / heads;
        const int head = block.kv_head * heads + flat - token * heads;
        const int64_t out_row = static_cast<int64_t>(block.q_row0) + token;
        const float down = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int64_t at = out_row * a.out_stride + static_cast<int64_t>(head) * D + ((warp * Q + q) * 4 + (lane >> 3)) * 4;
            if (!mine) continue;
            if (p.out_wide) {
                *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + at) =
                    make_uint2(pack_bf16x2(v[q].x * down, v[q].y * down), pack_bf16x2(v[q].z * down, v[q].w * down));
            } else {
                store_value(a.out, at, true, v[q].x * down);
                store_value(a.out, at + 1, true, v[q].y * down);
                store_value(a.out, at + 2, true, v[q].z * down);
                store_value(a.out, at + 3, true, v[q].w * down);
            }
        }
        if (warp == 0 && lane < 8 && mine && a.lse)
            a.lse[out_row * a.heads + head] = sum == 0.0f ? ninf : (top + log2f(sum)) * kLn2;
        __syncthreads();  // the item's shared values have been read
    }
}

// Blocks that can have at most so many tiles are not split: what the search
// for parts and the joining kernel take (4 us) is a tenth of such a block's
// time.
constexpr int kWholeTiles = 32;

int tile_sms() { return std::min(std::max(device_sm_count(), 2), kMaxTileCtas); }
size_t parts_bytes(int sms) { return (sizeof(TileHeader) + sms * sizeof(TileParts) + 255) / 256 * 256; }

// Keys that a block of so many rows can see.
int64_t key_bound(const KvCache &c, const AttnArgs &a, int rows) {
    return std::min(a.table_width << c.page_shift, a.window > 0 && a.causal ? int64_t{a.window} + rows : INT64_MAX);
}

template <int D>
int64_t tile_blocks(const KvCache &c, const AttnArgs &a) {
    const int64_t heads = a.heads / c.kv_heads;
    return ((a.total_q * heads + Tile<D>::rows - 1) / Tile<D>::rows + a.batch) * c.kv_heads;
}

template <int D>
cudaError_t launch_tiles(const KvCache &c, const AttnArgs &a, cudaStream_t stream, const LaunchCtx &ctx) {
    using T = Tile<D>;
    static int limits[kMaxDevices];
    constexpr size_t smem = 2 * T::stages * T::bytes + sizeof(TileShared) + 1024;
    static_assert(smem <= 232448, "shared memory per CTA");
    cudaError_t e = ensure_smem(attn_tile_kernel<D>, smem, false, limits);
    if (e != cudaSuccess) return e;
    TileParams p = {};
    p.a = a;
    p.k_codes = static_cast<const uint8_t *>(c.k_codes);
    p.k_scales = static_cast<const uint8_t *>(c.k_scales);
    p.v_codes = static_cast<const uint8_t *>(c.v_codes);
    p.v_scales = static_cast<const uint8_t *>(c.v_scales);
    p.num_pages = static_cast<int>(c.num_pages);
    p.page_shift = c.page_shift;
    p.kv_heads = c.kv_heads;
    const int q_size = a.q_bf16 ? 2 : 4;
    p.q_wide = reinterpret_cast<uintptr_t>(a.q) % 16 == 0 && a.q_stride * q_size % 16 == 0;
    p.out_wide = reinterpret_cast<uintptr_t>(a.out) % 16 == 0 && a.out_stride * 2 % 16 == 0;
    p.ctx = ctx;
    // splitting is left out where no block can have many tiles
    const int sms = tile_sms();
    const int64_t blocks = tile_blocks<D>(c, a);
    int64_t ctas = blocks;
    if (key_bound(c, a, T::rows) > kWholeTiles * kKeys) {
        p.split = sms;
        ctas = 4 * blocks <= 3 * sms ? sms : blocks + sms / 2;
    }
    p.header = static_cast<TileHeader *>(a.workspace);
    p.parts = reinterpret_cast<TileParts *>(p.header + 1);
    p.records = reinterpret_cast<float *>(static_cast<uint8_t *>(a.workspace) + parts_bytes(sms));
    e = launch_kernel(attn_tile_kernel<D>, dim3(static_cast<unsigned>(ctas)), dim3(T::threads), smem, stream, 1, p);
    if (e != cudaSuccess || p.split == 0) return e;
    return launch_kernel(attn_tile_join_kernel<D>, dim3(sms * 4), dim3(Join<D>::warps * 32), 0, stream, 1, p);
}

}  // namespace

// The streaming form works on 8 query rows of a request and key head at a
// time, this one on 128 or 256, whether they are there or not.  Picoseconds
// that a tile of 64 keys costs the whole GPU in either form:
//   head_dim 256  stream 3000, tiles 9500;  128  1400, 11500;  64  850, 10200
// and 9 us that this form takes longer to begin and end.  They follow from
// (us per call, two key heads, stream / tiles):
//   head_dim 256, one request: 64 rows with 4000 keys 30 / 40, with 32000
//   60 / 58, 512 rows with 32000 223 / 75, 2048 rows with 32000 788 / 208;
//   64 requests with 4000 keys: 16 rows 93 / 112, 32 rows 116 / 110, 64 rows
//   193 / 111, and 32 rows of one key head 83 / 64
//   head_dim 128: 64 rows of 64 requests with 4000 keys 96 / 119, 256 rows with
//   32000 keys 78 / 51;  head_dim 64, the same two: 68 / 107, 56 / 44
// The requests' lengths are not known here: the table's width stands for
// them, and their rows are taken to be alike.
bool attn_tiles_pay(const KvCache &c, const AttnArgs &a) {
    if (!a.out_bf16 || tile_blocks<256>(c, a) > INT32_MAX - kMaxTileCtas) return false;
    const int64_t group = a.heads / c.kv_heads, rows = c.head_dim == 256 ? Tile<256>::rows : Tile<128>::rows;
    const int64_t each = (a.total_q * group + a.batch - 1) / a.batch, most = a.max_q * group;
    const int64_t groups = a.batch * ((each + 7) / 8);
    const int64_t blocks = std::max(a.batch * ((each + rows - 1) / rows), a.batch - 1 + (most + rows - 1) / rows);
    const double stream = c.head_dim == 256 ? 3000 : c.head_dim == 128 ? 1400 : 850;
    const double tiles = c.head_dim == 256 ? 9500 : c.head_dim == 128 ? 11500 : 10200;
    const double keys = static_cast<double>(c.kv_heads) * static_cast<double>(key_bound(c, a, static_cast<int>(rows))) / kKeys;
    return keys * (static_cast<double>(groups) * stream - static_cast<double>(blocks) * tiles) > 9e6;
}

size_t attn_tiles_workspace_bytes() {
    const int sms = tile_sms();
    return parts_bytes(sms) + static_cast<size_t>(sms) * kPartFloats * sizeof(float);
}

cudaError_t launch_attn_tiles(const KvCache &c, const AttnArgs &a, cudaStream_t stream, const LaunchCtx &ctx) {
    if (c.head_dim == 64) return launch_tiles<64>(c, a, stream, ctx);
    if (c.head_dim == 128) return launch_tiles<128>(c, a, stream, ctx);
    return launch_tiles<256>(c, a, stream, ctx);
}

}  // namespace qmm
