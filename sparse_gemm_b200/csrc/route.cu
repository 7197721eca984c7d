// route.cu -- router of an expert layer: the k largest of each token's logits, their
// scores as weights, the (token, choice) pairs sorted by expert, and the gradient
// of the logits.
//
//     softmax: s_i = exp(l_i - m) / sum_j exp(l_j - m)     sigmoid: s_i = 1 / (1 + exp(-l_i))
//     w_j = factor s_{e_j}, or factor s_{e_j} / sum_i s_{e_i}
//
// A warp owns a token and keeps its logits in registers, 32 apart; a choice is a
// maximum over the warp (of the logit's bits, ordered as numbers) and a minimum
// over the experts that have it, so that ties go to the lowest one.  Choices go
// by the logits, whose order the scores share, so rounded scores decide nothing.
// Sigmoids that are divided by their sum are taken over exp(m), m the largest chosen
// logit or 0, exp(l - m) / (1 + exp(l)): far below 0, where the sigmoids themselves are
// no fp32 numbers, their quotients still are.
//
// Sorting is by counting: each CTA counts the experts of its run of tokens, and a
// second kernel adds up the counts of the runs before its own and places its
// pairs, whose rank among equals comes from match_any; every place is a sum of
// counts, so nothing depends on the order in which CTAs run.  Few tokens take
// one CTA and one kernel.  Launches and latency bound all of it.
#include <type_traits>

#include "common.cuh"
#include "grouped.cuh"
#include "internal.h"

namespace bsl {
namespace {

constexpr int kSmallTokens = 128;  // at most: one CTA routes and sorts them
constexpr int kSortWarps = 8;

struct RouteArgs {
    const void *logits;
    const float *dweights;
    const int32_t *chosen;  // backward
    int32_t *experts;
    float *weights;
    int32_t *offsets, *order, *counts;
    void *dlogits;
    int32_t T, E, k, run;  // run: tokens of a CTA
    int32_t half, sigmoid, renormalize;
    float factor;
};

// Logit i of a row, -inf past the last one.
__device__ __forceinline__ float logit(const RouteArgs &a, int64_t row, int i)
{
    if (i >= a.E) return -INFINITY;
    if (!a.half) return load_float(static_cast<const float *>(a.logits) + row * a.E + i);
    uint16_t w;
    asm volatile("ld.global.u16 %0, [%1];"
                 : "=h"(w)
                 : "l"(__cvta_generic_to_global(static_cast<const uint16_t *>(a.logits) + row * a.E + i)));
    return __uint_as_float(static_cast<uint32_t>(w) << 16);
}

// Bits in the order of the numbers: 0 for what is out, 1 for a NaN, -0 as 0.
__device__ __forceinline__ uint32_t key_of(float l)
{
    if (l != l) return 1;
    const uint32_t b = __float_as_uint(l + 0.f);
    return b >> 31 ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

__device__ __forceinline__ float sigmoid_of(float l) { return 1.f / (1.f + expf(-l)); }

// A row whose largest chosen logit is below this has sigmoids under 10^-304, and weights of zero.
constexpr float kNothing = -700.f;

// The same over exp(base), base = min(the largest chosen logit, 0); l is chosen.
__device__ __forceinline__ float sigmoid_over(float l, float base)
{
    return l > 0.f ? sigmoid_of(l) : expf(l - base) / (1.f + expf(l));
}

// A token's choices: lane j < k returns expert j and its weight.
template <int NE>
__device__ __forceinline__ void choose(const RouteArgs &a, int64_t row, int lane, int &expert, float &weight)
{
    float l[NE];
    uint32_t key[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) l[i] = logit(a, row, 32 * i + lane);
#pragma unroll
    for (int i = 0; i < NE; ++i) key[i] = 32 * i + lane < a.E ? key_of(l[i]) : 0;
    expert = 0;
    float mine = 0.f, top = 0.f;  // the chosen logit, the largest
    for (int j = 0; j < a.k; ++j) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < NE; ++i) best = max(best, key[i]);
        best = __reduce_max_sync(0xffffffffu, best);
        uint32_t at = 0xffffffffu;
#pragma unroll
        for (int i = NE - 1; i >= 0; --i)
            if (key[i] == best) at = 32 * i + lane;
        at = __reduce_min_sync(0xffffffffu, at);
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if (32 * i + lane == static_cast<int>(at)) {
                v = l[i];
                key[i] = 0;
            }
        v = __shfl_sync(0xffffffffu, v, at & 31);
        if (j == 0) top = v;
        if (lane == j) {
            expert = static_cast<int>(at);
            mine = v;
        }
    }
    float s = 0.f, total = 1.f;
    if (a.sigmoid) {
        if (a.renormalize) {
            if (lane < a.k && !(top < kNothing)) s = sigmoid_over(mine, fminf(top, 0.f));
            total = warp_sum(s);
        } else if (lane < a.k) {
            s = sigmoid_of(mine);
        }
    } else {
        float all = 0.f;
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if (32 * i + lane < a.E) all += expf(l[i] - top);
        all = warp_sum(all);
        if (lane < a.k) s = expf(mine - top);
        total = a.renormalize ? warp_sum(s) : all;
        if (all != all) total = all;  // a NaN or an infinity anywhere in the row
        if (top == -INFINITY) s = 0.f, total = 1.f;  // nothing is left: weights of zero
    }
    if (total == 0.f) total = 1.f;  // (sigmoids that are nothing)
    weight = a.factor * (s / total);
}

// Places of a run's `n` pairs (their experts in ids) among the pairs sorted by expert; base[e]: place of the run's
// first pair of expert e.  hist [kSortWarps][E] and rank [n] are scratch.  By the first kSortWarps warps of the
// block, all of which come here.
__device__ __forceinline__ void place_pairs(const RouteArgs &a, int64_t first, int n, const int32_t *ids, const int32_t *base,
                                            int32_t *hist, uint16_t *rank)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per = (n + 32 * kSortWarps - 1) / (32 * kSortWarps) * 32;  // pairs of a warp
    for (int i = threadIdx.x; i < kSortWarps * a.E; i += blockDim.x) hist[i] = 0;
    __syncthreads();
    if (warp < kSortWarps)
        for (int i = 0; i < per; i += 32) {
            const int p = warp * per + i + lane;
            const bool in = p < n;
            const int e = in ? ids[p] : -1;
            const uint32_t same = __match_any_sync(0xffffffffu, e);
            int seen = 0;
            if (in) {
                seen = hist[warp * a.E + e];
                rank[p] = static_cast<uint16_t>(seen + __popc(same & ((1u << lane) - 1u)));
            }
            __syncwarp();
            if (in && __ffs(same) - 1 == lane) hist[warp * a.E + e] = seen + __popc(same);
            __syncwarp();
        }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        int at = base[e];
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
            const int c = hist[w * a.E + e];
            hist[w * a.E + e] = at;
            at += c;
        }
    }
    __syncthreads();
    for (int p = threadIdx.x; p < n; p += blockDim.x)
        a.order[hist[p / per * a.E + ids[p]] + rank[p]] = static_cast<int32_t>(first + p);
}

// Shared memory of both kernels: counts or bases [E + 1], then what place_pairs needs.
struct RouteSmem {
    int32_t *count, *ids, *hist;
    uint16_t *rank;
    __device__ __forceinline__ RouteSmem(uint8_t *p, int E, int pairs)
    {
        count = reinterpret_cast<int32_t *>(p);
        hist = count + E + 1;
        ids = hist + kSortWarps * E;
        rank = reinterpret_cast<uint16_t *>(ids + pairs);
    }
    static size_t bytes(int E, int pairs) { return 4 * (static_cast<size_t>(E) + 1 + kSortWarps * E) + 6 * static_cast<size_t>(pairs); }
};

// Threads of k_route: a CTA that counts or sorts has up to 128 tokens, and latency bounds a token, so that many warps
// share them (16384 tokens, 128 experts: 8 warps 35 us, 32 warps 17).
constexpr int route_threads(int NE, int sort) { return sort == 0 ? 256 : NE >= 16 ? 512 : 1024; }

// Choices of a run of tokens; kSort 1: with their counts for k_sort, 2: and sorted here (one CTA).
template <int NE, int kSort>
__global__ void __launch_bounds__(route_threads(NE, kSort)) k_route(const RouteArgs a)
{
    extern __shared__ __align__(16) uint8_t smem[];
    const RouteSmem m(smem, a.E, a.run * a.k);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    dependents_may_launch();
    if (kSort) {
        for (int e = threadIdx.x; e <= a.E; e += blockDim.x) m.count[e] = 0;
        __syncthreads();
    }
    wait_for_prior_grid();
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * a.run;
    const int rows = static_cast<int>(a.T - row0 < a.run ? a.T - row0 : a.run);
    for (int r = warp; r < rows; r += blockDim.x / 32) {
        int expert;
        float weight;
        choose<NE>(a, row0 + r, lane, expert, weight);
        if (lane < a.k) {
            const int64_t p = (row0 + r) * a.k + lane;
            a.experts[p] = expert;
            a.weights[p] = weight;
            if (kSort) atomicAdd(&m.count[expert], 1);
            if (kSort == 2) m.ids[r * a.k + lane] = expert;
        }
    }
    if (kSort == 0) return;
    __syncthreads();
    if (kSort == 1) {
        for (int e = threadIdx.x; e < a.E; e += blockDim.x) a.counts[static_cast<int64_t>(blockIdx.x) * a.E + e] = m.count[e];
        return;
    }
    if (warp == 0) tile_starts(a.E, m.count, [&](int e) { return m.count[e]; });
    __syncthreads();
    for (int e = threadIdx.x; e <= a.E; e += blockDim.x) a.offsets[e] = m.count[e];
    place_pairs(a, 0, rows * a.k, m.ids, m.count, m.hist, m.rank);
}

__global__ void __launch_bounds__(512) k_sort(const RouteArgs a)
{
    extern __shared__ __align__(16) uint8_t smem[];
    const RouteSmem m(smem, a.E, a.run * a.k);
    const int warp = threadIdx.x >> 5;
    int32_t *before = m.hist;  // of this run, until place_pairs takes the memory
    dependents_may_launch();
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) m.count[e] = before[e] = 0;
    __syncthreads();
    wait_for_prior_grid();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * a.run * a.k;
    const int64_t left = static_cast<int64_t>(a.T) * a.k - first;
    const int n = static_cast<int>(left < a.run * a.k ? left : a.run * a.k);
    for (int p = threadIdx.x; p < n; p += blockDim.x) m.ids[p] = static_cast<int>(load_global(reinterpret_cast<const uint32_t *>(a.experts + first + p)));
    // counts of all runs, several threads an expert
    const int runs = gridDim.x, parts = blockDim.x / a.E > 1 ? blockDim.x / a.E : 1;
    for (int i = threadIdx.x; i < a.E * parts; i += blockDim.x) {
        const int e = i % a.E, part = i / a.E;
        int all = 0, prior = 0;
        const int end = (part + 1) * runs / parts;
        for (int c0 = part * runs / parts; c0 < end; c0 += 16) {  // sixteen loads on the way
            int v[16];
#pragma unroll
            for (int j = 0; j < 16; ++j)
                v[j] = c0 + j < end ? static_cast<int>(load_global(reinterpret_cast<const uint32_t *>(
                                          a.counts + static_cast<int64_t>(c0 + j) * a.E + e)))
                                    : 0;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                all += v[j];
                prior += c0 + j < static_cast<int>(blockIdx.x) ? v[j] : 0;
            }
        }
        if (all) atomicAdd(&m.count[e], all);
        if (prior) atomicAdd(&before[e], prior);
    }
    __syncthreads();
    if (warp == 0) tile_starts(a.E, m.count, [&](int e) { return m.count[e]; });
    __syncthreads();
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e <= a.E; e += blockDim.x) a.offsets[e] = m.count[e];
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) m.count[e] += before[e];
    __syncthreads();
    place_pairs(a, first, n, m.ids, m.count, m.hist, m.rank);
}

// dl of a token, from D_i = the sum of dw_j over the choices j of expert i, and G = sum_i D_i s_i:
//   softmax, weights s:          factor s_i (D_i - G)
//   softmax, weights s / S:      factor s_i / S (D_i - G / S) for the chosen, S = the sum of their scores
//   sigmoid:                     factor s_i (1 - s_i) D_i, or factor s_i (1 - s_i) (D_i - G / S) / S for the chosen,
//                                whose scores may all be over the same number
// Nothing is read by a choice's index, so one out of range does no harm.
template <int NE>
__global__ void __launch_bounds__(256) k_route_backward(const RouteArgs a)
{
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    dependents_may_launch();
    wait_for_prior_grid();
    if (row >= a.T) return;
    float l[NE], s[NE], D[NE];
    bool in[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) l[i] = logit(a, row, 32 * i + lane);
    int id = -1;
    float g = 0.f;
    if (lane < a.k) {
        id = static_cast<int>(load_global(reinterpret_cast<const uint32_t *>(a.chosen + row * a.k + lane)));
        g = load_float(a.dweights + row * a.k + lane);
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) D[i] = 0.f, in[i] = false;
    for (int j = 0; j < a.k; ++j) {
        const int e = __shfl_sync(0xffffffffu, id, j);
        const float d = __shfl_sync(0xffffffffu, g, j);
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if (32 * i + lane == e) D[i] += d, in[i] = true;
    }
    float slope[NE];  // of a score by its own logit, over the score's share
    if (a.sigmoid) {
        float top = 0.f;  // divided by their sum: over exp(base), as in the forward
        if (a.renormalize) {
            top = -INFINITY;
#pragma unroll
            for (int i = 0; i < NE; ++i)
                if (in[i]) top = fmaxf(top, l[i]);
#pragma unroll
            for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        }
        const float base = fminf(top, 0.f);
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const float small = expf(-fabsf(l[i])), one = 1.f / (1.f + small);
            const float e = top < kNothing ? 0.f : base < 0.f && in[i] ? expf(l[i] - base) : small;
            s[i] = l[i] >= 0.f ? one : e * one;
            slope[i] = e * one * one;
            if (l[i] != l[i]) s[i] = slope[i] = l[i];
        }
    } else {
        float top = -INFINITY, all = 0.f;
#pragma unroll
        for (int i = 0; i < NE; ++i) top = fmaxf(top, l[i]);
#pragma unroll
        for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            s[i] = 32 * i + lane < a.E && top != -INFINITY ? expf(l[i] - top) : 0.f;
            all += s[i];
        }
        all = warp_sum(all);
        if (all == 0.f) all = 1.f;  // nothing is left
#pragma unroll
        for (int i = 0; i < NE; ++i) s[i] = slope[i] = s[i] / all;
    }
    float G = 0.f, S = 0.f;
#pragma unroll
    for (int i = 0; i < NE; ++i) S += in[i] ? s[i] : 0.f;
    S = warp_sum(S);
    if (S == 0.f) S = 1.f;
    // divided by their sum: G / S, by the quotients, of which an only choice's is one, so that its difference is zero
#pragma unroll
    for (int i = 0; i < NE; ++i)
        if (in[i]) G += D[i] * (a.renormalize ? s[i] / S : s[i]);  // (a NaN that was not chosen is nobody's)
    G = warp_sum(G);
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = 32 * i + lane;
        if (e >= a.E) continue;
        float d;
        if (a.renormalize) d = in[i] ? slope[i] / S * (D[i] - G) : 0.f;
        else if (a.sigmoid) d = in[i] ? slope[i] * D[i] : 0.f;
        else d = slope[i] * (D[i] - G);
        d *= a.factor;
        if (a.half) static_cast<__nv_bfloat16 *>(a.dlogits)[row * a.E + e] = __float2bfloat16(d);
        else static_cast<float *>(a.dlogits)[row * a.E + e] = d;
    }
}

// Tokens of a CTA: all of a few, else as many as make 128 CTAs, 128 at most; of very many as many as make 1024 CTAs,
// since each CTA of k_sort reads all the others' counts, and as its memory holds (128 experts, 8 choices, 2^18 tokens: 574 us
// with 2048 runs, 328 with 1024; 2^20 tokens 5751 with 8192, 933 with 1024; 2^17 tokens 207).
constexpr int kMostRuns = 1024, kMostPairs = 8192;
int run_of(int32_t T, int32_t k)
{
    if (T <= kSmallTokens) return T;
    const int run = (T + 127) / 128;
    if (run <= kSmallTokens) return run < 8 ? 8 : run;
    const int many = static_cast<int>((static_cast<int64_t>(T) + kMostRuns - 1) / kMostRuns), most = kMostPairs / k;
    return many < kSmallTokens ? kSmallTokens : many < most ? many : most;
}
static_assert(kMostPairs / BSL_ROUTE_MAX_K >= kSmallTokens && kMostPairs <= 65535, "runs that grow, ranks of 16 bits");

template <int NE>
bsl_status route_of(RouteArgs &a, int sort, cudaStream_t s)
{
    const unsigned runs = static_cast<unsigned>((static_cast<int64_t>(a.T) + a.run - 1) / a.run);
    const size_t smem = sort ? RouteSmem::bytes(a.E, a.run * a.k) : 0;
    const unsigned threads = a.T > 8 ? route_threads(NE, sort) : 256;
    auto kern = sort == 0 ? k_route<NE, 0> : sort == 1 ? k_route<NE, 1> : k_route<NE, 2>;
    if (smem > 48 * 1024) {
        const bsl_status sa = set_smem_once(reinterpret_cast<const void *>(kern), 100 * 1024);
        if (sa != BSL_OK) return sa;
    }
    return cuda_status(launch_dependent(kern, runs, threads, smem, s, a));
}

template <typename F>
bsl_status by_width(int E, F f)
{
    if (E <= 32) return f(std::integral_constant<int, 1>());
    if (E <= 64) return f(std::integral_constant<int, 2>());
    if (E <= 128) return f(std::integral_constant<int, 4>());
    if (E <= 256) return f(std::integral_constant<int, 8>());
    if (E <= 512) return f(std::integral_constant<int, 16>());
    return f(std::integral_constant<int, 32>());
}

}  // namespace

size_t route_workspace_bytes(int32_t T, int32_t E, int32_t k)
{
    if (T <= kSmallTokens) return 0;
    const int run = run_of(T, k);
    return (static_cast<size_t>(T) + run - 1) / run * E * 4;
}

bsl_status launch_route(const void *logits, bool half, int32_t T, int32_t E, int32_t k, bool sigmoid, bool renormalize,
                        float factor, int32_t *experts, float *weights, int32_t *offsets, int32_t *order, void *workspace,
                        cudaStream_t s)
{
    RouteArgs a = {};
    a.logits = logits;
    a.experts = experts;
    a.weights = weights;
    a.offsets = offsets;
    a.order = order;
    a.counts = static_cast<int32_t *>(workspace);
    a.T = T;
    a.E = E;
    a.k = k;
    a.run = order ? run_of(T, k) : 8;
    a.half = half;
    a.sigmoid = sigmoid;
    a.renormalize = renormalize;
    a.factor = factor;
    const int sort = !order ? 0 : T <= kSmallTokens ? 2 : 1;
    const bsl_status st = by_width(E, [&](auto n) { return route_of<decltype(n)::value>(a, sort, s); });
    if (st != BSL_OK || sort != 1) return st;
    const size_t smem = RouteSmem::bytes(E, a.run * k);
    if (smem > 48 * 1024) {
        const bsl_status sa = set_smem_once(reinterpret_cast<const void *>(&k_sort), 100 * 1024);
        if (sa != BSL_OK) return sa;
    }
    return cuda_status(launch_dependent(k_sort, static_cast<unsigned>((static_cast<int64_t>(T) + a.run - 1) / a.run), 512, smem, s, a));
}

bsl_status launch_route_backward(const float *dweights, const void *logits, bool half, int32_t T, int32_t E, int32_t k,
                                 const int32_t *experts, bool sigmoid, bool renormalize, float factor, void *dlogits,
                                 cudaStream_t s)
{
    RouteArgs a = {};
    a.logits = logits;
    a.dweights = dweights;
    a.chosen = experts;
    a.dlogits = dlogits;
    a.T = T;
    a.E = E;
    a.k = k;
    a.half = half;
    a.sigmoid = sigmoid;
    a.renormalize = renormalize;
    a.factor = factor;
    return by_width(E, [&](auto n) {
        return cuda_status(launch_dependent(k_route_backward<decltype(n)::value>, static_cast<unsigned>((static_cast<int64_t>(T) + 7) / 8), 256, 0, s, a));
    });
}

}  // namespace bsl
