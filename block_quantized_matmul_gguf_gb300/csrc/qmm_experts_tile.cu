// qmm_experts_tile.cu -- the experts' Q4_0 products for many rows an expert
// (prompts, batches of requests), bf16 in and out, on tcgen05 tiles.
//
// Mathematics.  Y^T = W_e X_e^T for each expert e and the rows X_e of its pairs, which a
// first kernel writes in the pairs' order.  A weight w = (n - 8) d has 14 bits and enters
// as two bf16 parts of 8 bits each that add up to it (weights_of), which are two
// products into the same accumulator: each product is exact, for any scale, and sums
// are fp32 in tensor memory.  One binary16 part would take half the products (GeGLU of
// 2047 tokens 184 us for 122), but rounds each weight by up to 2^-12 of it and holds none
// of scales above 8188.
//
// Structure: one persistent CTA an SM; an item is 128 weight rows (64 gate and the same
// 64 up rows for GeGLU) by up to 128 of an expert's rows: tcgen05.mma.cta_group::1 with
// M = 128, the weights in tensor memory, x in shared memory.  An expert's rows are cut
// into equal tiles of a multiple of 32, so that the instruction's N follows the rows that
// are there.  Two accumulators: one is read out while the next item's products run.
//   warps 0, 3  x, every other stage each: boxes of 64 and 32 rows x 64 values, a lane each
//   warp 1      MMA, issued by the whole warp's elected lane
//   warp 2      weights as they are: boxes of 64 or 128 rows x 144 bytes
//   warps 28-31 the same where K is no multiple of 256 and rows lie on no 16 bytes:
//               the pieces of 16 that hold them, by cp.async, 32 rows a warp (GeGLU of 64
//               experts of 1024 x 2016, 2047 tokens: 195 us, where K of 2048 takes 182;
//               with one warp for all rows and weights in one part 203 for four warps'
//               147, and with a bulk copy a row, as TMA wants a request for each, 592)
//   warps 4-11  epilogue, two for each quarter of the lanes
//   warps 12-27 dequantisers: TMEM lanes 32 (w % 4) .., one stage (64 of K) of every
//               chunk (256 of K).  The first block's weights are formed in registers
//               before their slot is waited for, so that a free slot is filled at once.
// The pairs that a word of codes gives without a permutation are values 0 and 2, 1 and
// 3, so x is written in that order of K too.
// Which items (expert, tile, row block) there are depends on expert_start: each CTA
// forms the prefix sums of the experts' tiles in shared memory, and every role finds
// its CTA's items in them by two ballots.
// Every wait is bounded, as in the prefill GEMM.
//
// Bound, for prompts, by the tensor cores, at work 79 % of the time, 71 to 91 by SM
// (8 out of 64 experts of 1024 x 2048, 2047 tokens: 182 us with 14 for the rows,
// 1.51 PFLOP/s of products over all; without the low parts 134).  With few rows an expert by
// the hand-overs of its stages, no one of which is the bound (128 tokens: 54 us; without the
// low parts 50, without the weights' arithmetic 49, with an eighth of the products 47).
#include "qmm_internal.h"
#include "qmm_tc.cuh"

#include <algorithm>

namespace qmm {
namespace {

constexpr int BW = 128;      // weight rows of a CTA
constexpr int BT = 128;      // rows of x in a tile, at most
constexpr int BK = 64;       // K of a swizzle row of x
constexpr int CK = 256;      // K of a chunk: eight blocks
constexpr int SK = 128;      // K of a stage of x
constexpr int AK = 64;       // K of a stage of weights
constexpr int SUBS = SK / BK;
constexpr int A_SLOTS = 4, X_SLOTS = 4;  // stages in flight
static_assert(AK == BK && CK / AK == A_SLOTS, "a set of dequantisers keeps to one slot");
constexpr int X_SUB_BYTES = BT * BK * 2, X_SLOT_BYTES = SUBS * X_SUB_BYTES;
// A chunk of a row of weights is 144 bytes.  Where K is a multiple of 256 every row
// begins on 16 bytes and TMA copies boxes of them (WHOLE).  Otherwise the 16-byte
// pieces that hold them are copied, each row behind its own skew.
constexpr int RAW_CHUNK = 144;
template <bool WHOLE>
struct Raw {
    static constexpr int slots = WHOLE ? 4 : 3;  // chunks in flight
    static constexpr int pieces = 10;            // of 16 bytes, for 144 and a skew of up to 14
    static constexpr int row = WHOLE ? RAW_CHUNK : 176;  // 176: 8 rows in different banks, as 144
    static constexpr int slot_bytes = BW * row;
};
constexpr uint32_t D_COLS = 2 * BT, A_COLS = AK, TMEM_COLS = 512;  // two accumulators; two parts of the weights
static_assert(X_SLOTS % 2 == 0 && CK / SK % 2 == 0, "two x warps");
static_assert(D_COLS + A_SLOTS * A_COLS <= TMEM_COLS, "tensor memory");

constexpr int WARP_X = 0, WARP_MMA = 1, WARP_RAW = 2, WARP_X1 = 3, WARP_EPI = 4, EPI_WARPS = 8, WARP_DEQ = 12, DEQ_WARPS = 16;
constexpr int WARP_COPY = WARP_DEQ + DEQ_WARPS, COPY_WARPS = BW / 32;  // not WHOLE: warps that copy weights
template <bool WHOLE>
constexpr int kTileThreads = (WARP_COPY + (WHOLE ? 0 : COPY_WARPS)) * 32;
constexpr int X_WIDE = 64, X_BOX = 32;  // rows of a copy of x: as many wide ones as fit, and one more for the rest

template <bool WHOLE>
struct Layout {
    static constexpr int RAW_SLOTS = Raw<WHOLE>::slots;
    static constexpr int x = 0;
    static constexpr int raw = X_SLOTS * X_SLOT_BYTES;
    static constexpr int bars = raw + RAW_SLOTS * Raw<WHOLE>::slot_bytes;
    static constexpr int x_full = 0, x_empty = x_full + X_SLOTS, a_full = x_empty + X_SLOTS, a_empty = a_full + A_SLOTS,
                         raw_full = a_empty + A_SLOTS, raw_empty = raw_full + RAW_SLOTS, d_full = raw_empty + RAW_SLOTS,
                         d_empty = d_full + 2, final = d_empty + 2, nbars = final + 1;
    static constexpr int tmem_slot = bars + nbars * 8;
    static constexpr int abort_flag = tmem_slot + 4;
    static constexpr int cols = (abort_flag + 4 + 15) / 16 * 16;  // [4][BT] place in out of each column
    static constexpr int skew = cols + 4 * BT * 8;  // [RAW_SLOTS][32]: rows' skews repeat after 32
    static constexpr int tiles = skew + (WHOLE ? 0 : RAW_SLOTS * 128);  // Experts: four arrays of [experts + 1]
    static int total(int experts) { return tiles + (experts + 1) * 16 + 1024; }
};
static_assert(Layout<true>::tiles + (kMaxExperts + 1) * 16 + 1024 <= 232448 - 256 &&
                  Layout<false>::tiles + (kMaxExperts + 1) * 16 + 1024 <= 232448 - 256,
              "shared memory of a CTA");

constexpr int MOST_TILES = (1 << 30) - 1;  // where sums stop: above those of any plan, and twice it fits

struct TileParams {
    ExpertsPlan plan;
    void *out;           // GeGLU: h in bf16 by the pairs' order; down: z in fp32 by the pair
    int64_t out_stride;
    const uint8_t *w[2];  // not WHOLE: gate and up, or w[0]
    int64_t row_bytes;
    int n, chunks, blocks;  // chunks and blocks of K
    int row_blocks;      // of a matrix: of 128 rows (down) or 64 features
    uint32_t magic;      // 16, 16 in bf16, in a register
    bool even;           // out takes two neighbouring values at once
    LaunchCtx ctx;
};

// The experts' work, in shared memory: tiles in front of each expert's, its first
// pair, its pairs, and the rows of each of its tiles.
struct Experts {
    int *tiles, *start, *count, *per;
};

// An item: rows first .. first + cols - 1 of the sorted pairs of `expert`.  A CTA takes
// every gridDim.x-th item (tile, row block); whole warps step through them.
struct Item {
    int tile, row_block;
    int expert, first, cols, width;  // width: cols up to a multiple of 32
};

__device__ __forceinline__ int expert_count(const TileParams &p, int e, int &start) {
    const int64_t a = __ldcg(p.plan.expert_start + e), b = __ldcg(p.plan.expert_start + e + 1);
    if (a < 0 || b < a || b > p.plan.pairs_total) {
        record_error(p.ctx, kDevErrIndex);
        start = 0;
        return 0;
    }
    start = static_cast<int>(a);
    return static_cast<int>(b - a);
}

struct Items {
    int item, tile, row_block;      // the next one
    int tile_step, row_block_step;  // gridDim.x as tiles and row blocks
};
__device__ __forceinline__ Items items_from(const TileParams &p) {
    const int first = static_cast<int>(blockIdx.x), step = static_cast<int>(gridDim.x);
    Items at;
    at.item = first;
    at.tile = first / p.row_blocks;
    at.row_block = first - at.tile * p.row_blocks;
    at.tile_step = step / p.row_blocks;
    at.row_block_step = step - at.tile_step * p.row_blocks;
    return at;
}
// The next item, by a whole warp: two ballots find the expert.
__device__ __forceinline__ Item next_item(const TileParams &p, const Experts &ex, int lane, Items &at) {
    Item it;
    it.tile = at.tile;
    it.row_block = at.row_block;
    at.item += static_cast<int>(gridDim.x);
    at.tile += at.tile_step;
    at.row_block += at.row_block_step;
    if (at.row_block >= p.row_blocks) {
        at.row_block -= p.row_blocks;
        ++at.tile;
    }
    const int each = (p.plan.experts + 31) >> 5;
    int e = min(lane * each, p.plan.experts);
    const unsigned coarse = __ballot_sync(0xFFFFFFFFu, ex.tiles[e] <= it.tile);  // grows with e: lanes 0 .. some
    const int first = (31 - __clz(coarse)) * each;
    e = min(first + lane, p.plan.experts);
    const unsigned fine = __ballot_sync(0xFFFFFFFFu, lane < each && ex.tiles[e] <= it.tile);
    // experts without pairs share the place of the one behind them, which comes last
    it.expert = min(first + 31 - __clz(fine), p.plan.experts - 1);
    const int per = ex.per[it.expert], from = (it.tile - ex.tiles[it.expert]) * per;
    it.first = ex.start[it.expert] + from;
    it.cols = max(0, min(per, ex.count[it.expert] - from));
    it.width = max(32, (it.cols + 31) & ~31);
    return it;
}

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}

// A block's scale d in two parts of 5 bits each, and -24 times each (7 bits), as bf16
// pairs.  d has 11 bits; what rounding it to 5 leaves is a whole number of its last
// place from -32 to 32, which has 5 bits too.
struct Scale {
    uint32_t high, low, high24, low24;
};
__device__ __forceinline__ uint32_t twice(float v) { return __byte_perm(__float_as_uint(v), 0, 0x3232); }
__device__ __forceinline__ Scale scale_of(uint32_t half_bits) {
    const float d = half_bits_to_float(static_cast<uint16_t>(half_bits));
    const float high = __uint_as_float((__float_as_uint(d) + 0x40000u) & 0xFFF80000u), low = d - high;
    return Scale{twice(high), twice(low), twice(high * -24.0f), twice(low * -24.0f)};
}

// (n - 8) d of a word's eight codes in two parts: values 0 and 2, 1 and 3, 16 and 18,
// 17 and 19 of the block's quarter.  n - 8 has 3 bits (-8 one), so that each part
// has 8 and is exact in bf16; 16 + n is its code in the place of the upper mantissa
// bits of 16.
__device__ __forceinline__ void weights_of(uint32_t q, const Scale &d, uint32_t magic, uint32_t *high, uint32_t *low) {
    const uint32_t at[4] = {q << 3, q >> 5, q >> 1, q >> 9};  // bytes 0 and 2, 1 and 3: their lower codes, their upper ones
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t m = (at[i] & 0x00780078u) | magic;
        high[i] = fma_bf16x2(m, d.high, d.high24);
        low[i] = fma_bf16x2(m, d.low, d.low24);
    }
}

// Whether the phase of this parity is over, without waiting.
__device__ __forceinline__ bool test_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return ok != 0;
}

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
__device__ __forceinline__ void commit(uint32_t one, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(one)
        : "memory");
}
// 16 bytes, of which the first `bytes` are read and the others zeros
__device__ __forceinline__ void copy16_some(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// An arrival of this thread at the barrier once its copies so far are there.
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// 32 consecutive 32-bit columns of this thread's lane.
__device__ __forceinline__ void tmem_st_32cols(uint32_t taddr, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}

// D fp32, A and B bf16, both K-major, M = 128; N goes in at run time.
constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(BW >> 4) << 24);

// G: GeGLU.  A CTA's 128 accumulator rows are then 64 features: in lane quarter q,
// lanes 0-15 hold the gate rows of features 16q .. 16q+15, lanes 16-31 their up rows.
template <bool G, bool WHOLE>
__global__ void __launch_bounds__(kTileThreads<WHOLE>, 1)
    experts_tile_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_x64,
                        const __grid_constant__ CUtensorMap tmap_w,
                        const __grid_constant__ CUtensorMap tmap_w2, const __grid_constant__ TileParams p) {
    using Smem = Layout<WHOLE>;
    constexpr int RAW_SLOTS = Smem::RAW_SLOTS, RAW_ROW = Raw<WHOLE>::row, RAW_SLOT_BYTES = Raw<WHOLE>::slot_bytes;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = smem_addr(smem_raw);
    const uint32_t sbase = (raw_base + 1023u) & ~1023u;
    uint8_t *sgen = smem_raw + (sbase - raw_base);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const LaunchCtx ctx = p.ctx;

    auto bar = [&](uint32_t i) -> uint32_t { return sbase + Smem::bars + 8u * i; };
    int *abort_flag = reinterpret_cast<int *>(sgen + Smem::abort_flag);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sgen + Smem::tmem_slot);
    Experts ex;
    ex.tiles = reinterpret_cast<int *>(sgen + Smem::tiles);
    ex.start = ex.tiles + p.plan.experts + 1;
    ex.count = ex.start + p.plan.experts + 1;
    ex.per = ex.count + p.plan.experts + 1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < X_SLOTS; ++i) {
            mbar_init_addr(bar(Smem::x_full + i), 1);
            mbar_init_addr(bar(Smem::x_empty + i), 1);
        }
        for (int i = 0; i < A_SLOTS; ++i) {
            mbar_init_addr(bar(Smem::a_full + i), 4);  // a warp of each quarter
            mbar_init_addr(bar(Smem::a_empty + i), 1);
        }
        for (int i = 0; i < RAW_SLOTS; ++i) {
            mbar_init_addr(bar(Smem::raw_full + i), WHOLE ? 1 : COPY_WARPS * 32 + 1);  // each lane's copies, and the skews
            mbar_init_addr(bar(Smem::raw_empty + i), DEQ_WARPS);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init_addr(bar(Smem::d_full + i), 1);
            mbar_init_addr(bar(Smem::d_empty + i), EPI_WARPS);
        }
        mbar_init_addr(bar(Smem::final), 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == WARP_MMA) tmem_alloc_cta(sbase + Smem::tmem_slot, TMEM_COLS);
    // This kernel is launched behind the rows' kernel alone, each of whose threads lets it
    // begin only after its own wait for all that came before: what is older than the
    // rows is complete and in memory by now.  So the plan (read past L1) and the weights
    // (TMA) are taken at once, and only the warps that read rows or write
    // results wait for the rows' kernel: 128 tokens 43.4 -> 40.0 us.
    {  // tiles in front of each expert's
        __shared__ int32_t part[kTileThreads<WHOLE> / 32];
        const int per = (p.plan.experts + kTileThreads<WHOLE> - 1) / kTileThreads<WHOLE>;
        const int e0 = min(p.plan.experts, static_cast<int>(threadIdx.x) * per), e1 = min(p.plan.experts, e0 + per);
        int mine = 0, start;
        for (int e = e0; e < e1; ++e) mine += (expert_count(p, e, start) + BT - 1) / BT;
        int s = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, s, o);
            if (lane >= o) s = min(s + u, MOST_TILES);
        }
        if (lane == 31) part[warp] = s;
        __syncthreads();
        int before = s - mine;
        for (int w = 0; w < warp; ++w) before = min(before + part[w], MOST_TILES);
        for (int e = e0; e < e1; ++e) {
            const int count = expert_count(p, e, start);
            ex.tiles[e] = before;
            ex.start[e] = start;
            ex.count[e] = count;
            const int parts = (count + BT - 1) / BT;
            ex.per[e] = parts ? ((count + parts - 1) / parts + 31) & ~31 : 32;
            before = min(before + parts, MOST_TILES);
            if (e == p.plan.experts - 1) ex.tiles[p.plan.experts] = before;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t *>(tmem_slot);
    // a plan whose experts claim more than its pairs is not worked: sums stay exact
    const bool sound = ex.tiles[p.plan.experts] <= p.plan.pairs_total / BT + p.plan.experts;
    if (!sound && threadIdx.x == 0) record_error(ctx, kDevErrIndex);
    const int items = sound ? ex.tiles[p.plan.experts] * p.row_blocks : 0;
    const int chunks = p.chunks;

    Items at = items_from(p);
    if (warp == WARP_X || warp == WARP_X1) {
        pdl_wait();
        const uint32_t which = warp != WARP_X;  // every other stage; an item has an even number of them
        uint32_t it = which;
        bool ok = true;
        while (ok && at.item < items) {
            const Item t = next_item(p, ex, lane, at);
            // rows behind cols are others', and dropped
            const int sub = lane & (SUBS - 1), row = (lane / SUBS) * X_WIDE;
            const bool wide = row + X_WIDE <= t.width, mine = row < t.width;
            const CUtensorMap *map = wide ? &tmap_x64 : &tmap_x;
            const uint32_t bytes = static_cast<uint32_t>(t.width) * SK * 2;
            for (int st = static_cast<int>(which); st < chunks * (CK / SK); st += 2, it += 2) {
                const uint32_t s = it % X_SLOTS, full = bar(Smem::x_full + s);
                if (!warp_wait_or_abort(bar(Smem::x_empty + s), ((it / X_SLOTS) & 1u) ^ 1u, abort_flag, ctx)) {
                    ok = false;
                    break;
                }
                if (lane == 0) mbar_expect_tx_addr(full, bytes);
                __syncwarp();
                if (mine)
                    tma_load_2d(sbase + Smem::x + s * X_SLOT_BYTES + sub * X_SUB_BYTES + row * BK * 2, map, st * SK + sub * BK,
                                t.first + row, full);
            }
        }
        if (lane == 0) {
            // all copies have come
            for (uint32_t s = which; s < X_SLOTS; s += 2)
                if (it > s) {
                    const uint32_t last = it - 2 - ((it - 2 - s) % X_SLOTS);
                    wait_drain(bar(Smem::x_full + s), (last / X_SLOTS) & 1u, ctx);
                }
        }
    } else if (WHOLE ? warp == WARP_RAW : warp >= WARP_COPY) {
        const int64_t w_bytes = p.plan.experts * p.row_bytes * p.n;
        const int rows32 = warp - WARP_COPY;  // not WHOLE: which 32 rows of the slot
        uint32_t it = 0;
        bool ok = true;
        while (ok && at.item < items) {
            const Item t = next_item(p, ex, lane, at);
            const int row0 = t.row_block * (G ? BW / 2 : BW);
            // A warp copies 32 rows, 10 pieces each, in ten steps.  A row's skew repeats after
            // 32 rows, whose bytes are a multiple of 16.  Rows behind the expert's are
            // another's or zeros, and dropped.
            const int64_t base = (static_cast<int64_t>(t.expert) * p.n + row0) * p.row_bytes;
            const int64_t first = base & ~int64_t(15);
            int window[Raw<WHOLE>::pieces];  // from first on
            auto place_of = [&](int i) { return (i * 32 + lane) / 10 * RAW_ROW + (i * 32 + lane) % 10 * 16; };
            const int skew = static_cast<int>(base + lane * p.row_bytes) & 15;
            if constexpr (!WHOLE) {
#pragma unroll
                for (int i = 0; i < Raw<WHOLE>::pieces; ++i) {
                    const int at32 = i * 32 + lane;
                    window[i] = static_cast<int>(((base + at32 / 10 * p.row_bytes) & ~int64_t(15)) - first) + at32 % 10 * 16;
                }
            }
            for (int c = 0; c < chunks; ++c, ++it) {
                const uint32_t s = it % RAW_SLOTS, full = bar(Smem::raw_full + s);
                if (!warp_wait_or_abort(bar(Smem::raw_empty + s), ((it / RAW_SLOTS) & 1u) ^ 1u, abort_flag, ctx)) {
                    ok = false;
                    break;
                }
                const uint32_t to = sbase + Smem::raw + s * RAW_SLOT_BYTES;
                if constexpr (WHOLE) {
                    if (lane == 0) {
                        const int wrow = t.expert * p.n + row0;
                        mbar_expect_tx_addr(full, RAW_SLOT_BYTES);
                        tma_load_2d(to, &tmap_w, c * RAW_CHUNK, wrow, full);
                        if constexpr (G) tma_load_2d(to + (BW / 2) * RAW_ROW, &tmap_w2, c * RAW_CHUNK, wrow, full);
                    }
                    __syncwarp();
                } else {
                    const uint8_t *w = p.w[G ? rows32 >> 1 : 0];
                    const int64_t more = first + (G ? rows32 & 1 : rows32) * 32 * p.row_bytes + c * RAW_CHUNK;
                    const uint32_t to32 = to + rows32 * 32 * RAW_ROW;
                    if (more + 32 * p.row_bytes + 176 <= w_bytes) {  // windows end below 31 rows + 176 bytes
                        const uint8_t *src = w + more;
#pragma unroll
                        for (int i = 0; i < Raw<WHOLE>::pieces; ++i) copy16(to32 + place_of(i), src + window[i]);
                    } else {
#pragma unroll 1
                        for (int i = 0; i < Raw<WHOLE>::pieces; ++i) {
                            const int at32 = i * 32 + lane;
                            const int64_t from = more + ((base + at32 / 10 * p.row_bytes) & ~int64_t(15)) - first + at32 % 10 * 16;
                            const int64_t left = w_bytes - from;
                            copy16_some(to32 + place_of(i), w + (left > 0 ? from : 0),
                                        left >= 16 ? 16u : left > 0 ? static_cast<uint32_t>(left) : 0u);
                        }
                    }
                    copies_arrive(full);
                    if (rows32 == 0) {
                        reinterpret_cast<int *>(sgen + Smem::skew)[s * 32 + lane] = skew;
                        __syncwarp();
                        if (lane == 0) mbar_arrive_addr(full);
                    }
                }
            }
        }
        if constexpr (!WHOLE) copies_wait();
        if (lane == 0)
            for (uint32_t s = 0; s < RAW_SLOTS; ++s)
                if (it > s) {
                    const uint32_t last = it - 1 - ((it - 1 - s) % RAW_SLOTS);
                    wait_drain(bar(Smem::raw_full + s), (last / RAW_SLOTS) & 1u, ctx);
                }
    } else if (warp == WARP_MMA) {
        // the whole warp, so that the operands are known to be the same for all lanes:
        // a thread on its own has to move each to the uniform registers that the
        // products take theirs from, and paces the pipeline by that
        const uint32_t one = elected(), tmem = __shfl_sync(0xFFFFFFFFu, tmem_base, 0);
        const uint32_t bars = __shfl_sync(0xFFFFFFFFu, bar(0), 0);
        const uint64_t bdesc0 = sw128_desc(__shfl_sync(0xFFFFFFFFu, sbase, 0) + Smem::x);
        const int stages = __shfl_sync(0xFFFFFFFFu, chunks * (CK / SK), 0);
        auto desc_of = [&](const Item &t) {
            return kIdesc | static_cast<uint32_t>(__shfl_sync(0xFFFFFFFFu, t.width, 0) >> 3) << 17;
        };
        // both barriers of a stage of x at once: each look that succeeds takes some 100 cycles
        auto look = [&](uint32_t i) {
            return test_wait(bar(Smem::x_full + i % X_SLOTS), (i / X_SLOTS) & 1u) &&
                   test_wait(bar(Smem::a_full + 2 * i % A_SLOTS), (2 * i / A_SLOTS) & 1u);
        };
        uint32_t tiles_done = 0, it = 0;
        bool ok = true, issued = false;
        while (ok && at.item < items) {
            const uint32_t idesc = desc_of(next_item(p, ex, lane, at));
            const uint32_t d = tiles_done & 1u;  // accumulator
            if (!warp_wait_or_abort(bar(Smem::d_empty + d), ((tiles_done >> 1) & 1u) ^ 1u, abort_flag, ctx)) break;
            for (int st = 0; st < stages; ++st, ++it) {
                const uint32_t xs = it % X_SLOTS;
                if (!__all_sync(0xFFFFFFFFu, look(it))) {
                    ok = warp_wait_or_abort(bar(Smem::x_full + xs), (it / X_SLOTS) & 1u, abort_flag, ctx) &&
                         warp_wait_or_abort(bar(Smem::a_full + 2 * it % A_SLOTS), (2 * it / A_SLOTS) & 1u, abort_flag, ctx);
                    if (!ok) break;
                }
                const uint32_t to = tmem + d * BT;
                const uint64_t b = bdesc0 + xs * (X_SLOT_BYTES >> 4);
#pragma unroll
                for (int h = 0; h < SUBS; ++h) {
                    const uint32_t w = SUBS * it + h, as = w % A_SLOTS, a = tmem + D_COLS + as * A_COLS;
                    if (h > 0) {
                        ok = warp_wait_or_abort(bar(Smem::a_full + as), (w / A_SLOTS) & 1u, abort_flag, ctx);
                        if (!ok) break;
                    }
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < AK / 16; ++k) {  // the low part first
                        const uint64_t bk = b + h * (X_SUB_BYTES >> 4) + 2 * k;
                        product(one, to, a + 16 * k + 8, bk, idesc, k != 0 || h != 0 || st != 0);
                        product(one, to, a + 16 * k, bk, idesc, 1);
                    }
                    issued = true;
                    commit(one, bars + 8u * (Smem::a_empty + as));
                }
                if (!ok) break;
                commit(one, bars + 8u * (Smem::x_empty + xs));
            }
            if (ok) commit(one, bars + 8u * (Smem::d_full + d));
            ++tiles_done;
        }
        if (issued) {  // all products are done before tensor memory is freed
            commit(one, bars + 8u * Smem::final);
            wait_drain(bar(Smem::final), 0, ctx);
        }
    } else if (warp >= WARP_DEQ && warp < WARP_COPY) {
        // one stage of every chunk: two blocks of K
        const int q = warp & 3, part = (warp - WARP_DEQ) >> 2;
        const int row = G ? (lane >> 4) * (BW / 2) + q * 16 + (lane & 15) : q * 32 + lane;
        const uint32_t to = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + D_COLS + part * A_COLS;
        const int ctas = static_cast<int>(gridDim.x), first = static_cast<int>(blockIdx.x);
        const uint32_t total = first < items ? static_cast<uint32_t>((items - first + ctas - 1) / ctas) * chunks : 0u;
        const uint32_t place = static_cast<uint32_t>(row) * RAW_ROW + 36u * part;
        int c = 0;  // chunk of its item
        for (uint32_t it = 0; it < total; ++it) {
            const uint32_t r = it % RAW_SLOTS;
            if (!warp_wait_or_abort(bar(Smem::raw_full + r), (it / RAW_SLOTS) & 1u, abort_flag, ctx)) break;
            // two blocks are nine words; the first's codes begin in the middle of one
            const uint8_t *from = sgen + Smem::raw + r * RAW_SLOT_BYTES + place;
            uint32_t wd[9];
            if constexpr (WHOLE) {
                const uint32_t *src = reinterpret_cast<const uint32_t *>(from);
#pragma unroll
                for (int i = 0; i < 9; ++i) wd[i] = src[i];
            } else {
                const int skew = reinterpret_cast<const int *>(sgen + Smem::skew)[r * 32 + (row & 31)];  // even
                const uint32_t *src = reinterpret_cast<const uint32_t *>(from + (skew & ~3));
                const uint32_t which = skew & 2 ? 0x5432u : 0x3210u;
                uint32_t last = src[0];
#pragma unroll
                for (int i = 0; i < 9; ++i) {
                    const uint32_t next = src[i + 1];
                    wd[i] = __byte_perm(last, next, which);
                    last = next;
                }
                const int behind = p.blocks - 8 * c - 2 * part;  // blocks of K from here on
                // no weights behind K: codes are finite, so a scale of 0 takes them out
                if (behind <= 0) wd[0] &= 0xFFFF0000u;
                if (behind <= 1) wd[4] &= 0x0000FFFFu;
                if (++c == chunks) c = 0;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_addr(bar(Smem::raw_empty + r));
            // columns of a block: 16 of K's high and low parts, the other 16's
            uint32_t v[32];
            const Scale d0 = scale_of(wd[0] & 0xFFFFu), d1 = scale_of(wd[4] >> 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t *at = v + (i >> 1) * 16 + (i & 1) * 4;
                weights_of(__byte_perm(wd[i], wd[i + 1], 0x5432), d0, p.magic, at, at + 8);
            }
            if (!warp_wait_or_abort(bar(Smem::a_empty + part), (it & 1u) ^ 1u, abort_flag, ctx)) break;
            tc_fence_after();
            tmem_st_32cols(to, v);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t *at = v + (i >> 1) * 16 + (i & 1) * 4;
                weights_of(wd[5 + i], d1, p.magic, at, at + 8);
            }
            tmem_st_32cols(to + A_COLS / 2, v);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_addr(bar(Smem::a_full + part));
        }
    } else if (warp >= WARP_EPI && warp < WARP_DEQ) {
        const int q = warp & 3, part = (warp - WARP_EPI) >> 2;  // the two warps of a quarter take every other 32 columns
        const bool odd = lane & 1, upper = lane >= 16;
        uint64_t *table = reinterpret_cast<uint64_t *>(sgen + Smem::cols) + q * BT;
        uint32_t tiles_done = 0;
        pdl_wait();
        while (at.item < items) {
            const Item t = next_item(p, ex, lane, at);
            const uint32_t d = tiles_done & 1u;
            // lanes 2i and 2i + 1 exchange halves of two columns: each then has two
            // neighbouring features f, f + 1 of one
            const int f = t.row_block * (G ? BW / 2 : BW) + (G ? q * 16 + (lane & 14) : q * 32 + (lane & 30));
            for (int c = 32 * part + lane; c < t.width; c += 64) {  // place in out (none: 0)
                uint64_t to = 0;
                if (c < t.cols) {
                    const int pr = p.plan.pairs[t.first + c];
                    if (pr >= 0 && pr < p.plan.pairs_total)
                        to = reinterpret_cast<uint64_t>(p.out) + (G ? t.first + c : pr) * p.out_stride * (G ? 2 : 4);
                    else
                        record_error(ctx, kDevErrIndex);
                }
                table[c] = to;
            }
            __syncwarp();
            if (!warp_wait_or_abort(bar(Smem::d_full + d), (tiles_done >> 1) & 1u, abort_flag, ctx)) break;
            tc_fence_after();
            auto put = [&](uint64_t to, float lo, float hi) {
                if (to == 0 || f >= p.n) return;
                if constexpr (G) {
                    uint16_t *at = reinterpret_cast<uint16_t *>(to) + f;
                    const uint32_t v = pack_bf16x2(lo, hi);
                    if (p.even) {
                        *reinterpret_cast<uint32_t *>(at) = v;
                    } else {
                        at[0] = static_cast<uint16_t>(v);
                        if (f + 1 < p.n) at[1] = static_cast<uint16_t>(v >> 16);
                    }
                } else {
                    float *at = reinterpret_cast<float *>(to) + f;
                    if (p.even) {
                        *reinterpret_cast<float2 *>(at) = make_float2(lo, hi);
                    } else {
                        at[0] = lo;
                        if (f + 1 < p.n) at[1] = hi;
                    }
                }
            };
#pragma unroll 1
            for (int c = 32 * part; c < t.cols; c += 64) {
                uint32_t v[32];
                tmem_ld_32cols(tmem_base + d * BT + (static_cast<uint32_t>(q * 32) << 16) + c, v);
                if constexpr (G) {
                    // the lower lanes take columns 0-15, the upper ones 16-31
                    const int c0 = c + (lane & 16);
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        float h[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float other = __shfl_xor_sync(0xFFFFFFFFu, __uint_as_float(upper ? v[j + i] : v[16 + j + i]), 16);
                            const float g = upper ? other : __uint_as_float(v[j + i]);
                            const float u = upper ? __uint_as_float(v[16 + j + i]) : other;
                            h[i] = gelu_tanh_fast(g) * u;
                        }
                        const float got = __shfl_xor_sync(0xFFFFFFFFu, odd ? h[0] : h[1], 1);
                        put(table[c0 + j + odd], odd ? got : h[0], odd ? h[1] : got);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const float mine = __uint_as_float(odd ? v[j + 1] : v[j]);
                        const float got = __shfl_xor_sync(0xFFFFFFFFu, __uint_as_float(odd ? v[j] : v[j + 1]), 1);
                        put(table[c + j + odd], odd ? got : mine, odd ? mine : got);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_addr(bar(Smem::d_empty + d));
            ++tiles_done;
        }
    }

    pdl_launch_dependents();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == WARP_MMA) tmem_dealloc_cta(tmem_base, TMEM_COLS);
}

// Rows of x in the pairs' order, and of K in the weights': a warp a row.
// GeGLU: row i is x[pairs[i] / topk]; down: row i of h.  Bound by the bytes out.
struct RowsParams {
    ExpertsPlan plan;
    const uint16_t *x;
    int64_t x_stride;
    uint4 *rows;  // [pairs][padded / 8], zeros behind k
    int k, padded;
    bool gather;
    LaunchCtx ctx;
};

constexpr int kRowsWarps = 8;
constexpr int kRowsHeld = 8;  // 256 values each, loaded before the first is written

__global__ void __launch_bounds__(kRowsWarps * 32) experts_rows_kernel(const __grid_constant__ RowsParams p) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    // (the tile kernel relies on this order of the two, in every thread)
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kRowsWarps + (threadIdx.x >> 5); i < p.plan.pairs_total;
         i += static_cast<int64_t>(gridDim.x) * kRowsWarps) {
        int64_t from = i;
        if (p.gather) {
            const int pr = p.plan.pairs[i];
            if (pr < 0 || pr >= p.plan.pairs_total) continue;  // the products drop its column
            from = pr / p.plan.topk;
        }
        // eight c, of block c / 4: the values from 4 (c % 4) on and from 16 + 4 (c % 4) on
        const int all = p.k / 8, padded = p.padded / 8;  // padded: a multiple of 32
        const uint16_t *x = p.x + from * p.x_stride + (lane >> 2) * 32 + (lane & 3) * 4;
        uint4 *out = p.rows + i * padded;
        for (int c0 = 0; c0 < padded; c0 += kRowsHeld * 32) {
            uint2 a[kRowsHeld], b[kRowsHeld];
#pragma unroll
            for (int j = 0; j < kRowsHeld; ++j) {
                a[j] = b[j] = make_uint2(0, 0);
                if (c0 + j * 32 + lane < all) {
                    a[j] = *reinterpret_cast<const uint2 *>(x + (c0 + j * 32) * 8);
                    b[j] = *reinterpret_cast<const uint2 *>(x + (c0 + j * 32) * 8 + 16);
                }
            }
#pragma unroll
            for (int j = 0; j < kRowsHeld; ++j) {
                if (c0 + j * 32 >= padded) break;
                out[c0 + j * 32 + lane] = make_uint4(__byte_perm(a[j].x, a[j].y, 0x5410), __byte_perm(a[j].x, a[j].y, 0x7632),
                                                     __byte_perm(b[j].x, b[j].y, 0x5410), __byte_perm(b[j].x, b[j].y, 0x7632));
            }
        }
    }
}

int64_t padded_k(int64_t k) { return (k + CK - 1) / CK * CK; }
size_t rows_bytes(int64_t pairs, int64_t k) { return static_cast<size_t>(pairs) * 2 * padded_k(k); }

template <bool G, bool WHOLE>
cudaError_t launch_tile(const ExpertsPlan &plan, const uint8_t *w, const uint8_t *w2, const uint16_t *x, int64_t x_stride,
                        void *out, int64_t out_stride, int64_t n, int64_t k, void *workspace, cudaStream_t stream,
                        const LaunchCtx &ctx) {
    const int64_t padded = padded_k(k);
    uint16_t *xr = static_cast<uint16_t *>(workspace);
    CUtensorMap tx, tx64, tw = {}, tw2 = {};
    const uint64_t row = static_cast<uint64_t>(k / kQK) * kQ4_0Bytes, rows = static_cast<uint64_t>(plan.experts) * n;
    if (!encode_tmap_2d(&tx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, xr, padded, plan.pairs_total, padded * 2, BK, X_BOX, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tmap_2d(&tx64, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, xr, padded, plan.pairs_total, padded * 2, BK, X_WIDE, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    if (WHOLE && (!encode_tmap_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, w, row, rows, row, RAW_CHUNK, G ? BW / 2 : BW) ||
                  !encode_tmap_2d(&tw2, CU_TENSOR_MAP_DATA_TYPE_UINT8, G ? w2 : w, row, rows, row, RAW_CHUNK, G ? BW / 2 : BW)))
        return cudaErrorInvalidValue;
    const int tile_rows = G ? BW / 2 : BW;
    const TileParams p = {plan, out, out_stride, {w, G ? w2 : w}, static_cast<int64_t>(row), static_cast<int>(n),
                          static_cast<int>(padded / CK), static_cast<int>(k / kQK),
                          static_cast<int>((n + tile_rows - 1) / tile_rows), 0x41804180u,
                          n % 2 == 0 && out_stride % 2 == 0 && reinterpret_cast<uintptr_t>(out) % (G ? 4 : 8) == 0, ctx};
    static int limits[kMaxDevices];
    const size_t smem = Layout<WHOLE>::total(plan.experts);
    cudaError_t e = ensure_smem(experts_tile_kernel<G, WHOLE>, smem, false, limits);
    if (e != cudaSuccess) return e;
    const RowsParams r = {plan, x, x_stride, reinterpret_cast<uint4 *>(xr), static_cast<int>(k), static_cast<int>(padded), G, ctx};
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>((plan.pairs_total + kRowsWarps - 1) / kRowsWarps, int64_t(1) << 30));
    e = launch_kernel(experts_rows_kernel, dim3(grid), dim3(kRowsWarps * 32), 0, stream, 1, r);
    if (e != cudaSuccess) return e;
    return launch_kernel(experts_tile_kernel<G, WHOLE>, dim3(device_sm_count()), dim3(kTileThreads<WHOLE>), smem, stream, 1, tx, tx64,
                         tw, tw2, p);
}

}  // namespace

// Whether the tile form takes a product: bf16 in and out, rows of x in 16-byte
// pieces, and enough pairs an expert on average.
bool experts_tiles_pay(const ExpertsPlan &plan, const void *x, int64_t x_stride, bool bf16, int64_t n, int64_t k, bool geglu) {
    return bf16 && reinterpret_cast<uintptr_t>(x) % 16 == 0 && x_stride % 8 == 0 &&
           plan.experts * n < (int64_t(1) << 31) && experts_are_many(plan.pairs_total, plan.experts, k, geglu);
}

size_t experts_rows_bytes(int64_t pairs, int64_t k) { return rows_bytes(pairs, k); }

cudaError_t launch_experts_tile_geglu(const ExpertsGeglu &a, cudaStream_t stream, const LaunchCtx &ctx) {
    auto *launch = a.k % CK == 0 ? launch_tile<true, true> : launch_tile<true, false>;
    return launch(a.plan, a.wg, a.wu, static_cast<const uint16_t *>(a.x), a.x_stride, a.h, a.h_stride, a.n, a.k,
                  a.workspace, stream, ctx);
}

cudaError_t launch_experts_tile_down(const ExpertsDown &a, void *z, void *rows, cudaStream_t stream, const LaunchCtx &ctx) {
    auto *launch = a.k % CK == 0 ? launch_tile<false, true> : launch_tile<false, false>;
    return launch(a.plan, a.wd, nullptr, static_cast<const uint16_t *>(a.h), a.h_stride, z, a.n, a.n, a.k,
                  rows, stream, ctx);
}

}  // namespace qmm
