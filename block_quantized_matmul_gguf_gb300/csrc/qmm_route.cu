// qmm_route.cu -- experts of each token: scores, the choice of topk of them,
// their weights, and the (token, slot) pairs in the order of their experts
// (include/qmm.h, qmm_route).
//
// Mathematics.  s = softmax(l) or sigmoid(l), c = s + bias; the topk largest c
// among the kept groups, ties to the lowest index.  Without a bias c orders as
// l does, and the choice compares the logits themselves.  With one, c is
// formed in fp32 with an error that the comments bound; where compared values
// lie nearer than that allows, they are formed again in 64 bits.  So the choice is
// that of 64 bits everywhere, at the price of 32 (a token in some thousands takes the
// second way).
//
// A warp per token.  Each lane sorts its values as words of a key's upper bits and
// the expert's index, so that a round of the choice is one warp-wide maximum; a few
// more than topk are taken, ordered among themselves by their whole values, and
// the choice stands if the topk-th of them is clear of what was cut off (else the
// rounds are gone through with whole keys, in 64 bits).
//
// A pair's place is start[e] + the tokens before its own that chose e.  A token
// chooses an expert once at most, so within the tokens of a CTA that count is a
// population count over a bit mask per expert: no order of atomics enters.  Up
// to 512 tokens the CTAs are one cluster that passes its counts on through shared
// memory; beyond, clusters leave them in the workspace and a second launch places
// the pairs.
//
// Bound by latency for few tokens (one of 64 experts 4.2 us, 128 of 128 6.5), by
// instructions and their dependencies for many (some 500 a token with 256 experts:
// 8191 of them 29 us with the second launch, 53 % of the issue slots).
#include "qmm_internal.h"

#include <cooperative_groups.h>

#include <algorithm>

namespace qmm {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kSpan = 64;         // tokens of a bit mask, at most
constexpr int kMaxChunks = 256;   // CTAs: more tokens take more a CTA
constexpr int kMaxCluster = 8;
constexpr int kMore = 2;          // candidates beyond topk
constexpr float kInf = __builtin_huge_valf();

struct RouteParams {
    RouteArgs a;
    int64_t spans;     // per CTA
    int span;          // tokens of one
    unsigned group_magic;  // ceil(2^21 / experts of a group): e times it, shifted back, is e's group (e < 2^10)
    int chunks;        // CTAs, with those of the last cluster that have no tokens
    int cluster;       // CTAs of a cluster
    int32_t *hist;     // workspace: [clusters][experts] pairs of each expert, then [chunks][experts] those of the
                       // CTAs before in its cluster
    LaunchCtx ctx;
};

// Unsigned order of floats; NaN below -inf, 0 for what is not there.
__device__ __forceinline__ uint32_t order_of(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);  // -0 and 0 are equal
    if (v != v) return 1;
    return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ uint64_t order_of(double v) {
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
    if (v != v) return 1;
    return u ^ ((u >> 63) ? ~uint64_t(0) : uint64_t(1) << 63);
}

__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(0xFFFFFFFFu, v); }
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
    const uint32_t hi = __reduce_max_sync(0xFFFFFFFFu, static_cast<uint32_t>(v >> 32));
    const uint32_t lo = __reduce_max_sync(0xFFFFFFFFu, static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
    return static_cast<uint64_t>(hi) << 32 | lo;
}

__device__ __forceinline__ float load_logit(const float *row, int e) { return row[e]; }
__device__ __forceinline__ float load_logit(const uint16_t *row, int e) {
    return __uint_as_float(static_cast<uint32_t>(row[e]) << 16);
}

// The statistics of a token's scores.
struct Norm {
    float top, inv;  // softmax: the largest logit (0 where it is no finite number) and 1 / sum of exp(l - top), 0 for none
};

// A score as it is returned; the sigmoid by the exponential that does not overflow.
__device__ __forceinline__ float score_of(float l, const Norm &n, bool softmax) {
    if (softmax) return expf(l - n.top) * n.inv;
    const float e = expf(-fabsf(l));
    return (l < 0.0f ? e : 1.0f) / (1.0f + e);
}

// Below this a score is 0 in 64 bits, and counts as 0: log 2^-1075.
constexpr float kNoScore = -745.1332f;

// A chosen expert's score over some common factor, for a quotient by their sum: `most`
// is the chosen experts' largest logit.  The scores themselves may be too small for 32
// bits.  A softmax's are exp(l) but for a factor, and so are a sigmoid's, to 2^-92, where
// no logit is above -64.
__device__ __forceinline__ float relative_score(float l, float most, const Norm &n, bool softmax) {
    if (softmax && n.inv != n.inv) return n.inv;  // no number among the logits
    if (softmax ? l - n.top < kNoScore : l < kNoScore) return 0.0f;
    return softmax || most < -64.0f ? expf(l - most) : score_of(l, n, false);
}
// A score as it is compared; near values are formed again in 64 bits.
__device__ __forceinline__ float rough_score(float l, const Norm &n, bool softmax) {
    if (softmax) return __expf(l - n.top) * n.inv;
    const float z = -l > 80.0f ? 80.0f : -l;  // a NaN stays one
    return __fdividef(1.0f, 1.0f + __expf(z));
}

// The largest not yet taken of the warp's keys (element 32 j + lane): its key,
// and its index, the lowest of equals; it is taken.
template <int V, typename Key>
__device__ __forceinline__ Key take_largest(Key (&key)[V], int lane, int &index) {
    Key mine = key[0];
    int at = lane;
#pragma unroll
    for (int j = 1; j < V; ++j)
        if (key[j] > mine) {
            mine = key[j];
            at = 32 * j + lane;
        }
    const Key top = warp_max(mine);
    index = static_cast<int>(__reduce_min_sync(0xFFFFFFFFu, mine == top ? static_cast<unsigned>(at) : 0x7FFFFFFFu));
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (32 * j + lane == index) key[j] = 0;
    return top;
}

// The kept groups' mask from each group's score in lane g; `close` where the last
// kept and the first left lie within `near` of each other.
template <typename F>
__device__ __forceinline__ unsigned kept_groups(const RouteArgs &a, F total, F near, int lane, bool &close) {
    int rank = 0;  // the groups before this one
    for (int g = 0; g < a.groups; ++g) {
        const F other = __shfl_sync(0xFFFFFFFFu, total, g);
        rank += other > total || (other == total && g < lane);
    }
    close = false;
    if (a.group_topk < a.groups) {
        const unsigned in = __ballot_sync(0xFFFFFFFFu, lane < a.groups && rank == a.group_topk - 1);
        const unsigned out = __ballot_sync(0xFFFFFFFFu, lane < a.groups && rank == a.group_topk);
        const F least = __shfl_sync(0xFFFFFFFFu, total, __ffs(in) - 1), most = __shfl_sync(0xFFFFFFFFu, total, __ffs(out) - 1);
        close = !(least - most > near);
    }
    return __ballot_sync(0xFFFFFFFFu, lane < a.groups && rank < a.group_topk);
}

// Values of the experts into scratch ([experts], this warp's own), a NaN as -inf.
template <int V, typename F>
__device__ __forceinline__ void spread_values(const RouteArgs &a, const F (&c)[V], F *scratch, int lane) {
    __syncwarp();
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (32 * j + lane < a.experts) scratch[32 * j + lane] = c[j] == c[j] ? c[j] : static_cast<F>(-kInf);
    __syncwarp();
}

// The score of group `lane`: the sum of its group_best largest values.
template <typename F>
__device__ __forceinline__ F group_score(const RouteArgs &a, const F *scratch, int lane) {
    const int size = a.experts / a.groups;
    if (lane >= a.groups) return -kInf;
    F first = -kInf, second = -kInf;
    const F *v = scratch + lane * size;
    auto take = [&](F x) {
        second = max(second, min(first, x));
        first = max(first, x);
    };
    if (sizeof(F) == 4 && size % 4 == 0) {
        int i = lane % (size / 4);  // from another place in each lane: other banks
#pragma unroll 4
        for (int n = 0; n < size / 4; ++n) {
            const float4 x = reinterpret_cast<const float4 *>(v)[i];
            take(x.x), take(x.y), take(x.z), take(x.w);
            if (++i == size / 4) i = 0;
        }
    } else {
        int i = lane % size;
#pragma unroll 1
        for (int n = 0; n < size; ++n) {
            take(v[i]);
            if (++i == size) i = 0;
        }
    }
    const F total = a.group_best == 2 && size > 1 ? first + second : first;
    return total == total ? total : static_cast<F>(-kInf);  // of inf and -inf
}

template <int V, typename Key>
__device__ __forceinline__ void keep(const RouteParams &p, unsigned kept, Key (&key)[V], int lane) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const unsigned e = 32 * j + lane;
        const unsigned g = e * p.group_magic >> 21;  // e / size
        if (e < static_cast<unsigned>(p.a.experts) && !(kept >> g & 1)) key[j] = 0;
    }
}

// Descending order of V words.
template <int V>
__device__ __forceinline__ void sort_words(uint32_t (&w)[V]) {
    // odd-even merge sort
#pragma unroll
    for (int p = 1; p < V; p <<= 1)
#pragma unroll
        for (int k = p; k >= 1; k >>= 1)
#pragma unroll
            for (int j = k % p; j + k < V; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < V && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const uint32_t x = max(w[i + j], w[i + j + k]), y = min(w[i + j], w[i + j + k]);
                        w[i + j] = x;
                        w[i + j + k] = y;
                    }
}

// The choice by words of keys' upper bits and indexes: lane r < topk ends with
// the r-th id.  value, wide: of an expert, in fp32 and in 64 bits; false where the
// choice is not clear.
template <int V, typename Value, typename Wide>
__device__ __forceinline__ bool choose_by_words(const RouteArgs &a, const uint32_t (&key)[V], float near, bool exact, Value value,
                                                Wide wide, int lane, int &mine) {
    constexpr int kBits = V == 1 ? 5 : V == 2 ? 6 : V == 4 ? 7 : V == 8 ? 8 : V == 16 ? 9 : 10;
    constexpr uint32_t kIndex = (1u << kBits) - 1;
    uint32_t w[V];
#pragma unroll
    for (int j = 0; j < V; ++j) w[j] = key[j] ? (key[j] & ~kIndex) | (kIndex - (32 * j + lane)) : 0;
    sort_words<V>(w);
    const int taken = exact ? a.topk : min(a.topk + kMore, 32);
    uint32_t got = 0, last = 0;
    for (int r = 0; r < taken; ++r) {
        last = warp_max(w[0]);
        if (last == 0) break;  // none left
        if (lane == r) got = last;
        const bool hit = w[0] == last;
#pragma unroll
        for (int j = 0; j + 1 < V; ++j) w[j] = hit ? w[j + 1] : w[j];
        w[V - 1] = hit ? 0 : w[V - 1];
    }
    if (__popc(__ballot_sync(0xFFFFFFFFu, got != 0)) < a.topk) return false;  // what is no number has no word
    mine = static_cast<int>(kIndex - (got & kIndex));
    if (exact) return true;  // the words hold whole keys
    const float v = got ? value(mine) : 0.0f;
    const uint32_t whole = got ? order_of(v) : 0;
    // mostly the words' order is the values', and clear: lane r's neighbours, down to
    // the first that is not chosen, and what was cut off
    {
        const float before = __shfl_up_sync(0xFFFFFFFFu, v, 1);
        bool plain = got == 0 || lane > a.topk || (lane == 0 ? v == v : before - v > fmaxf(near, 0.0f));
        if (last != 0 && got != 0 && lane < a.topk)
            plain &= near < 0.0f ? whole > (last | kIndex) : v - value_of(last | kIndex) > near;
        if (__all_sync(0xFFFFFFFFu, plain)) return true;
    }
    // the candidates' own order
    int rank = 0;
    float above = kInf;  // the next larger value
    for (int r = 0; r < taken; ++r) {
        const uint32_t k = __shfl_sync(0xFFFFFFFFu, whole, r);
        const int i = __shfl_sync(0xFFFFFFFFu, mine, r);
        const bool before = k > whole || (k == whole && i < mine);
        rank += before;
        if (before) above = fminf(above, value_of(k));
    }
    // nothing that was cut off, which lies at `last` and its hidden bits at most, may
    // come near the chosen; `near` less than 0: values are exact
    bool clear = last == 0 || got == 0 || rank >= a.topk ||
                 (near < 0.0f ? whole > (last | kIndex) : v - value_of(last | kIndex) > near);
    if (!__all_sync(0xFFFFFFFFu, clear)) return false;
    // neighbours within `near`, down to the first that is not chosen, are compared
    // again in 64 bits
    clear = got == 0 || rank > a.topk || near < 0.0f || above - v > near;
    if (!__all_sync(0xFFFFFFFFu, clear)) {
        if (__any_sync(0xFFFFFFFFu, got != 0 && v != v)) return false;
        const double x = wide(mine, got != 0);
        rank = 0;
        for (int r = 0; r < taken; ++r) {
            const double other = __shfl_sync(0xFFFFFFFFu, x, r);
            const int i = __shfl_sync(0xFFFFFFFFu, mine, r);
            const bool is = __shfl_sync(0xFFFFFFFFu, got, r) != 0;
            rank += is && (other > x || (other == x && i < mine));
        }
    }
    // to the lanes of their ranks
    int id = 0;
    for (int r = 0; r < taken; ++r) {
        const int i = __shfl_sync(0xFFFFFFFFu, mine, r), k = __shfl_sync(0xFFFFFFFFu, got ? rank : 32, r);
        if (k == lane) id = i;
    }
    mine = id;
    return true;
}

// The sum of exp(l - top) of a token in 64 bits, by its warp.
template <typename T>
__device__ __noinline__ double wide_sum(const RouteArgs &a, const T *row, float top, int lane) {
    double sum = 0.0;
#pragma unroll 1
    for (int e = lane; e < a.experts; e += 32) sum += exp(static_cast<double>(load_logit(row, e)) - static_cast<double>(top));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    return sum;
}

// A value of the choice in 64 bits.
__device__ __forceinline__ double wide_value(const RouteArgs &a, float l, int e, const Norm &norm, double sum) {
    double s;
    if (a.score == 0) {
        const double w = exp(static_cast<double>(l) - static_cast<double>(norm.top));
        s = sum == 0.0 ? 0.0 : w / sum;
    } else {
        s = 1.0 / (1.0 + exp(-static_cast<double>(l)));
    }
    return a.bias ? s + static_cast<double>(a.bias[e]) : s;
}

// The kept groups again, from their best values in 64 bits.  `close` stays where a
// group's third value lies within `off` of its second, so that it is not known
// which those are.
template <typename T>
__device__ __noinline__ unsigned wide_groups(const RouteArgs &a, const T *row, const Norm &norm, const float *scratch, float off,
                                             int lane, bool &close) {
    const int size = a.experts / a.groups;
    const double sum = a.score == 0 ? wide_sum(a, row, norm.top, lane) : 0.0;
    double total = -kInf;
    bool unsure = false;
    if (lane < a.groups) {
        float v[3] = {-kInf, -kInf, -kInf};
        int at[2] = {0, 0};
        for (int i = 0; i < size; ++i) {
            const float x = scratch[lane * size + i];
            const int e = lane * size + i;
            if (x > v[0]) {
                v[2] = v[1], v[1] = v[0], v[0] = x;
                at[1] = at[0], at[0] = e;
            } else if (x > v[1]) {
                v[2] = v[1], v[1] = x, at[1] = e;
            } else if (x > v[2]) {
                v[2] = x;
            }
        }
        const int best = min(a.group_best, size);
        unsure = size > best && !(v[best - 1] - v[best] > off);
        if (v[best - 1] > -kInf) {
            total = wide_value(a, load_logit(row, at[0]), at[0], norm, sum);
            if (best == 2) total += wide_value(a, load_logit(row, at[1]), at[1], norm, sum);
        }
    }
    unsure = __any_sync(0xFFFFFFFFu, unsure);
    const unsigned kept = kept_groups<double>(a, total == total ? total : static_cast<double>(-kInf), 0.0, lane, close);
    close = unsure;
    return kept;
}

// The choice with all values whole, in 64 bits.
template <int V, typename T>
__device__ __noinline__ int choose_wide(const RouteParams &p, const T *row, const Norm &norm, double *scratch, int lane) {
    const RouteArgs &a = p.a;
    const double sum = a.score == 0 ? wide_sum(a, row, norm.top, lane) : 0.0;
    const bool scored = a.bias != nullptr || (a.groups > 1 && a.group_best == 2);
    double x[V];
    uint64_t key[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int e = 32 * j + lane;
        x[j] = 0.0;
        key[j] = 0;
        if (e < a.experts) {
            const float l = load_logit(row, e);
            x[j] = scored ? wide_value(a, l, e, norm, sum) : static_cast<double>(l);
            key[j] = order_of(a.bias ? x[j] : static_cast<double>(l));
        }
    }
    if (a.groups > 1) {
        bool close;
        spread_values<V, double>(a, x, scratch, lane);
        keep<V>(p, kept_groups<double>(a, group_score<double>(a, scratch, lane), 0.0, lane, close), key, lane);
    }
    int mine = 0;
    for (int r = 0; r < a.topk; ++r) {
        int index;
        take_largest<V, uint64_t>(key, lane, index);
        if (lane == r) mine = index;
    }
    return mine;
}

// One token's experts: lane r < topk ends with the r-th id.
template <int V, typename T>
__device__ __forceinline__ int choose(const RouteParams &p, const T *row, const Norm &norm, const float (&l)[V], char *scratch,
                                      int lane) {
    const RouteArgs &a = p.a;
    uint32_t key[V];
    const bool softmax = a.score == 0;
    const bool by_score = a.bias != nullptr;
    float near = -1.0f;
    bool close = false;
    if (by_score || (a.groups > 1 && a.group_best == 2)) {
        float c[V], largest = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int e = 32 * j + lane;
            const float b = by_score && e < a.experts ? a.bias[e] : 0.0f;
            c[j] = e < a.experts ? rough_score(l[j], norm, softmax) + b : -kInf;
            key[j] = e >= a.experts ? 0 : order_of(by_score ? c[j] : l[j]);
            if (e < a.experts && fabsf(c[j]) < kInf) largest = fmaxf(largest, fabsf(c[j]));
        }
        largest = __uint_as_float(warp_max(__float_as_uint(largest)));
        // Errors, in units of 2^-24.  Sigmoid: the argument's product with log2(e)
        // and the exponential leave 2 + |l| of exp(-l), which moves a score by at
        // most 1; sum and division add 4: a difference of two is off by less than
        // 16.  Softmax: product, exponential and division leave less than 8 of the
        // largest score (1 / sum); the sum's 47 are common to all, so that a
        // difference of two is off by 47 of it, again at most of the largest score.
        // Adding the bias rounds by 1 of the value.  A difference of two then lies
        // within `near`; a group's score is a sum of two, off by twice that.
        const float off = (softmax ? 64.0f * norm.inv : 16.0f) * 5.9604644775390625e-08f + 4.76837158203125e-07f * largest;
        if (by_score) near = off;
        if (a.groups > 1) {
            spread_values<V, float>(a, c, reinterpret_cast<float *>(scratch), lane);
            unsigned kept = kept_groups<float>(a, group_score<float>(a, reinterpret_cast<float *>(scratch), lane), 2.0f * off, lane, close);
            if (close) kept = wide_groups(a, row, norm, reinterpret_cast<float *>(scratch), off, lane, close);
            keep<V>(p, kept, key, lane);
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) key[j] = 32 * j + lane < a.experts ? order_of(l[j]) : 0;
        if (a.groups > 1) {  // by their best logit, exactly
            bool any;
            spread_values<V, float>(a, l, reinterpret_cast<float *>(scratch), lane);
            keep<V>(p, kept_groups<float>(a, group_score<float>(a, reinterpret_cast<float *>(scratch), lane), 0.0f, lane, any), key, lane);
        }
    }
    int mine = 0;
    if (!close) {
        const auto value = [&](int e) {
            const float x = load_logit(row, e);
            return by_score ? rough_score(x, norm, softmax) + a.bias[e] : x;
        };
        const auto wide = [&](int e, bool there) {
            const double sum = softmax ? wide_sum(a, row, norm.top, lane) : 0.0;
            return there ? wide_value(a, load_logit(row, e), e, norm, sum) : 0.0;
        };
        // a bf16 logit's last 16 bits are 0: words hold it whole
        if (choose_by_words<V>(a, key, near, sizeof(T) == 2 && !by_score, value, wide, lane, mine)) return mine;
    }
    return choose_wide<V, T>(p, row, norm, reinterpret_cast<double *>(scratch), lane);
}

// Exclusive prefix sum of n counts (n <= 2 kThreads) in shared memory, in
// place; returns the total.
__device__ __forceinline__ int block_prefix(int32_t *v, int n) {
    __shared__ int32_t part[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i = 2 * threadIdx.x;
    const int a = i < n ? v[i] : 0, b = i + 1 < n ? v[i + 1] : 0;
    int s = a + b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (lane >= o) s += u;
    }
    if (lane == 31) part[warp] = s;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += part[w];
        total += part[w];
    }
    if (i < n) v[i] = before + s - a - b;
    if (i + 1 < n) v[i + 1] = before + s - b;
    __syncthreads();
    return total;
}

// Where the pairs of `span` tokens go: base[e] + the tokens before in the span.
// ids: [span][topk], -1 where there is none.  base moves behind them.
__device__ __forceinline__ void place_span(const RouteArgs &a, int64_t token0, int span, const int32_t *ids, uint32_t (*mask)[2],
                                           int32_t *base) {
    const int n = span * a.topk;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const int t = i / a.topk, e = ids[i];
        const int64_t token = token0 + t;
        if (token >= a.tokens) break;
        const int64_t flat = token * a.topk + (i - t * a.topk);
        if (e < 0) {
            a.pairs[flat] = -1;  // tokens that are not there are the last ones
            continue;
        }
        const uint32_t lo = mask[e][0], hi = mask[e][1];
        const int before = t < 32 ? __popc(lo & ((1u << t) - 1)) : __popc(lo) + __popc(hi & ((1u << (t - 32)) - 1));
        a.pairs[base[e] + before] = static_cast<int32_t>(flat);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.experts; e += kThreads) base[e] += __popc(mask[e][0]) + __popc(mask[e][1]);
    __syncthreads();
}

// Tokens that are there.
__device__ __forceinline__ int64_t real_tokens(const RouteParams &p) {
    if (!p.a.count) return p.a.tokens;
    const int64_t n = *p.a.count;
    if ((n < 0 || n > p.a.tokens) && blockIdx.x == 0 && threadIdx.x == 0) record_error(p.ctx, kDevErrIndex);
    return n < 0 ? 0 : n > p.a.tokens ? p.a.tokens : n;
}

struct Shared {
    uint32_t (*mask)[2];  // [experts]
    int32_t *base;        // [experts]
    int32_t *count;       // [experts], this CTA's pairs
    int32_t *ids;         // [kSpan][topk]
    char *scratch;        // [kWarps][experts] doubles, groups only
};
__device__ __forceinline__ Shared shared_of(char *smem, const RouteArgs &a) {
    Shared s;
    s.scratch = smem;
    smem += a.groups > 1 ? static_cast<size_t>(kWarps) * a.experts * 8 : 0;
    s.mask = reinterpret_cast<uint32_t(*)[2]>(smem);
    smem += a.experts * 8;
    s.base = reinterpret_cast<int32_t *>(smem);
    smem += a.experts * 4;
    s.count = reinterpret_cast<int32_t *>(smem);
    smem += a.experts * 4;
    s.ids = reinterpret_cast<int32_t *>(smem);
    return s;
}

template <int V, typename T>
__global__ void __launch_bounds__(kThreads, V <= 8 ? 2 : 1) route_kernel(const __grid_constant__ RouteParams p) {
    extern __shared__ __align__(16) char smem[];
    const RouteArgs &a = p.a;
    const Shared s = shared_of(smem, a);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t real = real_tokens(p);
    for (int e = threadIdx.x; e < a.experts; e += kThreads) s.count[e] = 0;
    for (int64_t span = 0; span < p.spans; ++span) {
        const int64_t token0 = (blockIdx.x * p.spans + span) * p.span;
        for (int e = threadIdx.x; e < a.experts; e += kThreads) s.mask[e][0] = s.mask[e][1] = 0;
        __syncthreads();
        for (int t = warp; t < p.span && token0 + t < a.tokens; t += kWarps) {
            const int64_t token = token0 + t;
            int id = -1;
            float w = 0.0f;
            if (token < real) {
                const T *row = static_cast<const T *>(a.logits) + token * a.logits_stride;
                float l[V];
                float top = -kInf;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const int e = 32 * j + lane;
                    l[j] = e < a.experts ? load_logit(row, e) : -kInf;
                    top = fmaxf(top, l[j]);
                }
                Norm norm = {0.0f, 0.0f};
                if (a.score == 0) {
                    top = value_of(warp_max(order_of(top)));
                    norm.top = top == -kInf ? 0.0f : top;
                    float sum = 0.0f;
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        if (32 * j + lane < a.experts) sum += expf(l[j] - norm.top);
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
                    norm.inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                }
                id = choose<V, T>(p, row, norm, l, s.scratch + static_cast<size_t>(warp) * a.experts * 8, lane);
                const bool chosen = lane < a.topk;
                const float mine = chosen ? load_logit(row, id) : -kInf;
                if (!a.renormalize) {
                    w = chosen ? score_of(mine, norm, a.score == 0) : 0.0f;
                } else {
                    const float most = value_of(warp_max(order_of(mine)));
                    w = chosen ? relative_score(mine, most, norm, a.score == 0) : 0.0f;
                    float sum = w;
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
                    w = sum == 0.0f ? 0.0f : w / sum;
                }
                w *= a.scale;
                if (chosen) atomicOr(&s.mask[id][t >> 5], 1u << (t & 31));
            }
            if (lane < a.topk) {
                a.ids[token * a.topk + lane] = id;
                a.weights[token * a.topk + lane] = w;
                s.ids[t * a.topk + lane] = id;
            }
        }
        __syncthreads();
        for (int e = threadIdx.x; e < a.experts; e += kThreads) s.count[e] += __popc(s.mask[e][0]) + __popc(s.mask[e][1]);
    }
    // this CTA's share of its cluster's counts
    const cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
    const int rank = static_cast<int>(blockIdx.x) & (p.cluster - 1);  // a power of two
    if (p.cluster > 1)
        cluster.sync();
    else
        __syncthreads();
    const bool only = p.chunks == p.cluster;
    int before[2] = {0, 0};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int e = threadIdx.x + h * kThreads;
        if (e >= a.experts) break;
        int sum = 0;
        for (int c = 0; c < p.cluster; ++c) {
            const int n = p.cluster > 1 ? *cluster.map_shared_rank(s.count + e, c) : s.count[e];
            sum += n;
            if (c < rank) before[h] += n;
        }
        if (only) {
            s.base[e] = sum;
        } else {
            if (rank == 0) p.hist[static_cast<int64_t>(blockIdx.x / p.cluster) * a.experts + e] = sum;
            p.hist[static_cast<int64_t>(p.chunks / p.cluster + blockIdx.x) * a.experts + e] = before[h];
        }
    }
    if (only) {  // starts and places at once
        __syncthreads();
        const int total = block_prefix(s.base, a.experts);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int e = threadIdx.x + h * kThreads;
            if (e >= a.experts) break;
            if (blockIdx.x == 0) a.expert_start[e] = s.base[e];
            s.base[e] += before[h];
        }
        if (blockIdx.x == 0 && threadIdx.x == 0) a.expert_start[a.experts] = total;
        __syncthreads();
        place_span(a, static_cast<int64_t>(blockIdx.x) * p.span, p.span, s.ids, s.mask, s.base);
    }
    if (p.cluster > 1) cluster.sync();  // the others have read this CTA's counts
}

__global__ void __launch_bounds__(kThreads) place_kernel(RouteParams p) {
    extern __shared__ __align__(16) char smem[];
    RouteArgs a = p.a;
    a.groups = 1;  // no scratch here
    const Shared s = shared_of(smem, a);
    pdl_wait();
    pdl_launch_dependents();
    // pairs of each expert in all, and in front of this CTA's (in s.count): several
    // threads share an expert where there are more threads
    const int clusters = p.chunks / p.cluster, here = static_cast<int>(blockIdx.x) / p.cluster;
    for (int e = threadIdx.x; e < a.experts; e += kThreads) {
        s.base[e] = 0;
        s.count[e] = p.hist[static_cast<int64_t>(clusters + blockIdx.x) * a.experts + e];
    }
    __syncthreads();
    const int parts = max(1, kThreads / a.experts), each = (clusters + parts - 1) / parts;
    const int mine = threadIdx.x / a.experts;
    for (int e = parts > 1 ? threadIdx.x - mine * a.experts : threadIdx.x; e < a.experts && (parts == 1 || mine < parts); e += kThreads) {
        const int c0 = parts > 1 ? mine * each : 0, c1 = min(clusters, c0 + each);
        int sum = 0, before = 0;
#pragma unroll 16
        for (int c = c0; c < c1; ++c) {
            const int n = p.hist[static_cast<int64_t>(c) * a.experts + e];
            sum += n;
            if (c < here) before += n;
        }
        atomicAdd(&s.base[e], sum);  // whole numbers: in any order
        atomicAdd(&s.count[e], before);
    }
    __syncthreads();
    const int total = block_prefix(s.base, a.experts);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int e = threadIdx.x + h * kThreads;
        if (e >= a.experts) break;
        const int start = s.base[e];
        if (blockIdx.x == 0) a.expert_start[e] = start;
        s.base[e] = start + s.count[e];
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) a.expert_start[a.experts] = total;
    for (int64_t span = 0; span < p.spans; ++span) {
        const int64_t token0 = (blockIdx.x * p.spans + span) * p.span;
        if (token0 >= a.tokens) break;
        for (int e = threadIdx.x; e < a.experts; e += kThreads) s.mask[e][0] = s.mask[e][1] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < p.span * a.topk; i += kThreads) {
            const int t = i / a.topk;
            const int e = token0 + t < a.tokens ? a.ids[token0 * a.topk + i] : -1;
            s.ids[i] = e;
            if (e >= 0) atomicOr(&s.mask[e][t >> 5], 1u << (t & 31));
        }
        __syncthreads();
        place_span(a, token0, p.span, s.ids, s.mask, s.base);
    }
}

// How the tokens are shared out.  A warp takes up to four of a CTA's tokens one
// after another; clusters of a power of two, the last of whose CTAs may be
// without tokens.
void shape(int64_t tokens, RouteParams &p) {
    p.span = tokens <= kMaxCluster * 16 ? 16 : tokens <= kMaxChunks * 32 ? 32 : kSpan;
    if (tokens > kMaxCluster * 32 && tokens <= kMaxCluster * 64) p.span = 64;  // still one launch
    const int64_t all = (tokens + p.span - 1) / p.span;
    p.spans = (all + kMaxChunks - 1) / kMaxChunks;
    const int chunks = static_cast<int>((all + p.spans - 1) / p.spans);
    p.cluster = 1;
    while (p.cluster < chunks && p.cluster < kMaxCluster) p.cluster *= 2;
    p.chunks = (chunks + p.cluster - 1) / p.cluster * p.cluster;
}

size_t smem_bytes(const RouteArgs &a, bool scratch) {
    return (scratch && a.groups > 1 ? static_cast<size_t>(kWarps) * a.experts * 8 : 0) + a.experts * 16 + kSpan * a.topk * 4;
}

template <int V, typename T>
cudaError_t launch_v(const RouteParams &p, cudaStream_t stream) {
    static int limits[kMaxDevices];
    const size_t smem = smem_bytes(p.a, true);
    if (smem > 32 * 1024) {
        const cudaError_t e = ensure_smem(route_kernel<V, T>, smem, false, limits);
        if (e != cudaSuccess) return e;
    }
    return launch_kernel(route_kernel<V, T>, dim3(p.chunks), dim3(kThreads), smem, stream, p.cluster, p);
}

template <typename T>
cudaError_t launch_t(const RouteParams &p, cudaStream_t stream) {
    const int v = (p.a.experts + 31) / 32;
    return v <= 1   ? launch_v<1, T>(p, stream)
           : v <= 2 ? launch_v<2, T>(p, stream)
           : v <= 4 ? launch_v<4, T>(p, stream)
           : v <= 8 ? launch_v<8, T>(p, stream)
           : v <= 16 ? launch_v<16, T>(p, stream)
                     : launch_v<32, T>(p, stream);
}

}  // namespace

// Of a call with any number of tokens up to this one: the CTAs are most at 8192, and
// fewer again where a CTA takes more.
size_t route_workspace_bytes(int64_t tokens, int experts) {
    RouteParams p;
    shape(std::min<int64_t>(tokens, kMaxChunks * 32), p);
    return p.chunks == p.cluster ? 0 : static_cast<size_t>(p.chunks / p.cluster + p.chunks) * experts * sizeof(int32_t);
}

cudaError_t launch_route(const RouteArgs &args, cudaStream_t stream, const LaunchCtx &ctx) {
    RouteParams p;
    p.a = args;
    shape(args.tokens, p);
    const int size = args.experts / args.groups;
    p.group_magic = ((1u << 21) + size - 1) / size;
    p.hist = static_cast<int32_t *>(args.workspace);
    p.ctx = ctx;
    const cudaError_t e = args.bf16 ? launch_t<uint16_t>(p, stream) : launch_t<float>(p, stream);
    if (e != cudaSuccess || p.chunks == p.cluster) return e;
    static_assert(kMaxExperts * 16 + kSpan * kMaxTopk * 4 <= 48 * 1024, "place_kernel keeps to the default limit");
    const size_t place = smem_bytes(args, false);
    return launch_kernel(place_kernel, dim3(p.chunks), dim3(kThreads), place, stream, 1, p);
}

}  // namespace qmm
