// qmm_route.cu -- experts of each token: scores, the choice of topk of them,
// their weights, and the (token, slot) pairs in the order of their experts
// (include/qmm.h, qmm_route).
//
// Mathematics.  s = softmax(l) or sigmoid(l), c = s + bias; the topk largest c
// among the kept groups, ties to the lowest index.  Without a bias c orders as
// l does, and the choice compares the logits themselves.  With one, c is
// formed in fp32 with an error that the comments bound; where two of the
// compared values lie nearer than twice that bound, the token's scores are
// formed again in 64 bits.  So the choice is that of 64 bits everywhere, at the
// price of 32 (a token in some thousands takes the second way).
//
// A pair's place is start[e] + the tokens before its own that chose e.  A token
// chooses an expert once at most, so within 64 tokens that count is a
// population count over a bit mask per expert: no order of atomics enters.
//
// Bound by latency: a warp per token, 64 tokens a CTA.  Up to 64 tokens one
// launch does all; beyond, the CTAs leave their counts per expert in the
// workspace and a second launch places the pairs.
#include "qmm_internal.h"

#include <algorithm>

namespace qmm {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kSpan = 64;         // tokens of one bit mask
constexpr int kMaxChunks = 256;   // CTAs: more tokens take several spans a CTA
constexpr float kInf = __builtin_huge_valf();

struct RouteParams {
    RouteArgs a;
    int64_t spans;     // of kSpan tokens, per CTA
    int chunks;        // CTAs
    int32_t *hist;     // workspace: [chunks][experts] pairs of each expert
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

__device__ __forceinline__ float load_logit(const void *row, int e, bool bf16) {
    if (bf16) return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(row)[e]) << 16);
    return static_cast<const float *>(row)[e];
}

// The statistics of a token's scores.
struct Norm {
    float top, sum;  // softmax: the largest logit (0 where it is no finite number) and the sum of exp(l - top)
};

__device__ __forceinline__ float score_of(float l, const Norm &n, bool softmax) {
    if (!softmax) return 1.0f / (1.0f + expf(-l));
    return n.sum == 0.0f ? 0.0f : expf(l - n.top) / n.sum;
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

// Marks what lies in groups that are not kept: lane g scores group g by the
// sum of its `best` largest values (scratch: [experts], this warp's own).
// Returns whether the last kept and the first left group lie within `near` of
// each other; group scores of F stay exact enough for that by the caller.
template <int V, typename F, typename Key>
__device__ __forceinline__ bool keep_groups(const RouteArgs &a, const F (&c)[V], Key (&key)[V], F *scratch, int lane,
                                            F near) {
    const int size = a.experts / a.groups;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (32 * j + lane < a.experts) scratch[32 * j + lane] = c[j];
    __syncwarp();
    F first = -kInf, second = -kInf;
    bool none = true;
    if (lane < a.groups) {
        int i = lane % size;  // from another place in each lane: other banks
        for (int n = 0; n < size; ++n) {
            const F v = scratch[lane * size + i];
            if (v > first) {
                second = first;
                first = v;
            } else if (v > second) {
                second = v;
            }
            none &= v != v;
            if (++i == size) i = 0;
        }
    }
    F total = a.group_best == 2 && size > 1 ? first + second : first;
    if (none || total != total) total = -kInf;
    // a group's rank: the groups before it
    int rank = 0;
    bool close = false;
    for (int g = 0; g < a.groups; ++g) {
        const F other = __shfl_sync(0xFFFFFFFFu, total, g);
        rank += other > total || (other == total && g < lane);
    }
    const unsigned kept = __ballot_sync(0xFFFFFFFFu, lane < a.groups && rank < a.group_topk);
    if (a.group_topk < a.groups) {
        const unsigned in = __ballot_sync(0xFFFFFFFFu, lane < a.groups && rank == a.group_topk - 1);
        const unsigned out = __ballot_sync(0xFFFFFFFFu, lane < a.groups && rank == a.group_topk);
        const F least = __shfl_sync(0xFFFFFFFFu, total, __ffs(in) - 1), most = __shfl_sync(0xFFFFFFFFu, total, __ffs(out) - 1);
        close = !(least - most > near);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int e = 32 * j + lane;
        if (e < a.experts && !(kept >> (e / size) & 1)) key[j] = 0;
    }
    return close;
}

// One token's experts: lane r < topk ends with the r-th id.
template <int V>
__device__ __forceinline__ int choose(const RouteArgs &a, const void *row, const Norm &norm, const float (&l)[V], char *scratch,
                                      int lane) {
    uint32_t key[V];
    const bool softmax = a.score == 0;
    const bool by_score = a.bias != nullptr;
    float near = 0.0f, largest = 0.0f;
    bool close = false;
    if (by_score || (a.groups > 1 && a.group_best == 2)) {
        float c[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int e = 32 * j + lane;
            const float b = by_score && e < a.experts ? a.bias[e] : 0.0f;
            c[j] = e < a.experts ? score_of(l[j], norm, softmax) + b : -kInf;
            key[j] = e >= a.experts ? 0 : order_of(by_score ? c[j] : l[j]);
            if (e < a.experts && fabsf(c[j]) < kInf) largest = fmaxf(largest, fabsf(c[j]));
        }
        largest = value_of(warp_max(order_of(largest)));
        // Errors.  Sigmoid: expf (2 ulp), sum and division leave 5 * 2^-24 of
        // a score below 1.  Softmax: those and the argument's rounding leave
        // less than 8 * 2^-24 of the largest score (1 / sum), and the sum's
        // 40 * 2^-24 is common to all, so that a difference of two is off by
        // 40 * 2^-24 of it, again at most of the largest score.  Adding the
        // bias rounds by 2^-24 of the value.  A difference of two then lies
        // within `near`; a group's score is a sum of two, off by twice that.
        const float unit = softmax ? (norm.sum > 0.0f ? 3.814697265625e-06f / norm.sum : 0.0f) : 9.5367431640625e-07f;
        near = unit + 4.76837158203125e-07f * largest;
        if (a.groups > 1) close = keep_groups<V, float>(a, c, key, reinterpret_cast<float *>(scratch), lane, 2.0f * near);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) key[j] = 32 * j + lane < a.experts ? order_of(l[j]) : 0;
        if (a.groups > 1) {  // by their best logit, exactly
            float c[V];
#pragma unroll
            for (int j = 0; j < V; ++j) c[j] = l[j];
            keep_groups<V, float>(a, c, key, reinterpret_cast<float *>(scratch), lane, -1.0f);
        }
    }
    int mine = 0;
    if (!by_score) {
        if (!close) {
            for (int r = 0; r < a.topk; ++r) {
                int index;
                take_largest<V, uint32_t>(key, lane, index);
                if (lane == r) mine = index;
            }
            return mine;
        }
    } else if (!close) {
        // one more than is chosen: the last choice has to be clear too
        float before = kInf;
        for (int r = 0; r <= a.topk; ++r) {
            int index;
            const uint32_t top = take_largest<V, uint32_t>(key, lane, index);
            if (top == 0) break;  // none left
            const float v = value_of(top);
            close |= !(before - v > near);  // or no number
            before = v;
            if (r < a.topk && lane == r) mine = index;
        }
        if (!close) return mine;
    }
    // 64 bits
    double x[V], sum = 0.0;
    uint64_t wide[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int e = 32 * j + lane;
        const double v = e < a.experts ? static_cast<double>(load_logit(row, e, a.bf16)) : 0.0;
        x[j] = softmax ? exp(v - static_cast<double>(norm.top)) : 1.0 / (1.0 + exp(-v));
        if (e < a.experts) sum += x[j];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int e = 32 * j + lane;
        if (softmax) x[j] = sum == 0.0 ? 0.0 : x[j] / sum;
        if (by_score && e < a.experts) x[j] += static_cast<double>(a.bias[e]);
        wide[j] = e >= a.experts ? 0 : by_score ? order_of(x[j]) : order_of(static_cast<double>(load_logit(row, e, a.bf16)));
    }
    if (a.groups > 1) keep_groups<V, double>(a, x, wide, reinterpret_cast<double *>(scratch), lane, 0.0);
    for (int r = 0; r < a.topk; ++r) {
        int index;
        take_largest<V, uint64_t>(wide, lane, index);
        if (lane == r) mine = index;
    }
    return mine;
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

// Where the pairs of kSpan tokens go: base[e] + the tokens before in the span.
// ids: [kSpan][topk], -1 where there is none.  base moves behind them.
__device__ __forceinline__ void place_span(const RouteArgs &a, int64_t token0, const int32_t *ids, uint32_t (*mask)[2], int32_t *base) {
    const int n = kSpan * a.topk;
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
    s.ids = reinterpret_cast<int32_t *>(smem);
    return s;
}

template <int V>
__global__ void __launch_bounds__(kThreads) route_kernel(RouteParams p) {
    extern __shared__ __align__(16) char smem[];
    const RouteArgs &a = p.a;
    const Shared s = shared_of(smem, a);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t real = real_tokens(p);
    const bool one = p.chunks == 1;
    for (int e = threadIdx.x; e < a.experts; e += kThreads) s.base[e] = 0;
    for (int64_t span = 0; span < p.spans; ++span) {
        const int64_t token0 = (blockIdx.x * p.spans + span) * kSpan;
        for (int e = threadIdx.x; e < a.experts; e += kThreads) s.mask[e][0] = s.mask[e][1] = 0;
        __syncthreads();
        for (int t = warp; t < kSpan && token0 + t < a.tokens; t += kWarps) {
            const int64_t token = token0 + t;
            int id = -1;
            float w = 0.0f;
            if (token < real) {
                const void *row = a.bf16 ? static_cast<const void *>(static_cast<const uint16_t *>(a.logits) + token * a.logits_stride)
                                         : static_cast<const void *>(static_cast<const float *>(a.logits) + token * a.logits_stride);
                float l[V];
                float top = -kInf;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const int e = 32 * j + lane;
                    l[j] = e < a.experts ? load_logit(row, e, a.bf16) : -kInf;
                    top = fmaxf(top, l[j]);
                }
                Norm norm = {0.0f, 1.0f};
                if (a.score == 0) {
                    top = value_of(warp_max(order_of(top)));
                    norm.top = top == -kInf ? 0.0f : top;
                    float sum = 0.0f;
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        if (32 * j + lane < a.experts) sum += expf(l[j] - norm.top);
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
                    norm.sum = sum;
                }
                id = choose<V>(a, row, norm, l, s.scratch + static_cast<size_t>(warp) * a.experts * 8, lane);
                const bool chosen = lane < a.topk;
                w = chosen ? score_of(load_logit(row, id, a.bf16), norm, a.score == 0) : 0.0f;
                if (a.renormalize) {
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
        if (!one)
            for (int e = threadIdx.x; e < a.experts; e += kThreads) s.base[e] += __popc(s.mask[e][0]) + __popc(s.mask[e][1]);
    }
    if (!one) {
        for (int e = threadIdx.x; e < a.experts; e += kThreads) p.hist[static_cast<int64_t>(blockIdx.x) * a.experts + e] = s.base[e];
        return;
    }
    // the only span: starts and places at once
    for (int e = threadIdx.x; e < a.experts; e += kThreads) s.base[e] = __popc(s.mask[e][0]) + __popc(s.mask[e][1]);
    __syncthreads();
    const int total = block_prefix(s.base, a.experts);
    for (int e = threadIdx.x; e < a.experts; e += kThreads) a.expert_start[e] = s.base[e];
    if (threadIdx.x == 0) a.expert_start[a.experts] = total;
    place_span(a, 0, s.ids, s.mask, s.base);
}

__global__ void __launch_bounds__(kThreads) place_kernel(RouteParams p) {
    extern __shared__ __align__(16) char smem[];
    RouteArgs a = p.a;
    a.groups = 1;  // no scratch here
    const Shared s = shared_of(smem, a);
    pdl_wait();
    pdl_launch_dependents();
    // pairs of each expert in front of this CTA's, and in all
    int before[2] = {0, 0};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int e = threadIdx.x + h * kThreads;
        if (e >= a.experts) break;
        int sum = 0;
#pragma unroll 8
        for (int c = 0; c < p.chunks; ++c) {
            const int n = p.hist[static_cast<int64_t>(c) * a.experts + e];
            sum += n;
            if (c < static_cast<int>(blockIdx.x)) before[h] += n;
        }
        s.base[e] = sum;
    }
    __syncthreads();
    const int total = block_prefix(s.base, a.experts);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int e = threadIdx.x + h * kThreads;
        if (e >= a.experts) break;
        const int start = s.base[e];
        if (blockIdx.x == 0) a.expert_start[e] = start;
        s.base[e] = start + before[h];
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) a.expert_start[a.experts] = total;
    for (int64_t span = 0; span < p.spans; ++span) {
        const int64_t token0 = (blockIdx.x * p.spans + span) * kSpan;
        if (token0 >= a.tokens) break;
        for (int e = threadIdx.x; e < a.experts; e += kThreads) s.mask[e][0] = s.mask[e][1] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < kSpan * a.topk; i += kThreads) {
            const int t = i / a.topk;
            const int e = token0 + t < a.tokens ? a.ids[token0 * a.topk + i] : -1;
            s.ids[i] = e;
            if (e >= 0) atomicOr(&s.mask[e][t >> 5], 1u << (t & 31));
        }
        __syncthreads();
        place_span(a, token0, s.ids, s.mask, s.base);
    }
}

int chunks_of(int64_t tokens, int64_t &spans) {
    const int64_t all = (tokens + kSpan - 1) / kSpan;
    spans = std::max<int64_t>(1, (all + kMaxChunks - 1) / kMaxChunks);
    return static_cast<int>((all + spans - 1) / spans);
}

size_t smem_bytes(const RouteArgs &a, bool scratch) {
    return (scratch && a.groups > 1 ? static_cast<size_t>(kWarps) * a.experts * 8 : 0) + a.experts * 12 + kSpan * a.topk * 4;
}

template <int V>
cudaError_t launch_v(const RouteParams &p, cudaStream_t stream) {
    static int limits[kMaxDevices];
    const size_t smem = smem_bytes(p.a, true);
    if (smem > 32 * 1024) {
        const cudaError_t e = ensure_smem(route_kernel<V>, smem, false, limits);
        if (e != cudaSuccess) return e;
    }
    return launch_kernel(route_kernel<V>, dim3(p.chunks), dim3(kThreads), smem, stream, 1, p);
}

}  // namespace

size_t route_workspace_bytes(int64_t tokens, int experts) {
    int64_t spans;
    const int chunks = chunks_of(tokens, spans);
    return chunks > 1 ? static_cast<size_t>(chunks) * experts * sizeof(int32_t) : 0;
}

cudaError_t launch_route(const RouteArgs &args, cudaStream_t stream, const LaunchCtx &ctx) {
    RouteParams p;
    p.a = args;
    p.chunks = chunks_of(args.tokens, p.spans);
    p.hist = static_cast<int32_t *>(args.workspace);
    p.ctx = ctx;
    static int limits[kMaxDevices];
    const size_t place = smem_bytes(args, false);
    cudaError_t e = cudaSuccess;
    if (p.chunks > 1 && place > 32 * 1024) e = ensure_smem(place_kernel, place, false, limits);
    if (e != cudaSuccess) return e;
    const int v = (args.experts + 31) / 32;
    e = v <= 1   ? launch_v<1>(p, stream)
        : v <= 2 ? launch_v<2>(p, stream)
        : v <= 4 ? launch_v<4>(p, stream)
        : v <= 8 ? launch_v<8>(p, stream)
        : v <= 16 ? launch_v<16>(p, stream)
                  : launch_v<32>(p, stream);
    if (e != cudaSuccess || p.chunks == 1) return e;
    return launch_kernel(place_kernel, dim3(p.chunks), dim3(kThreads), place, stream, 1, p);
}

}  // namespace qmm
