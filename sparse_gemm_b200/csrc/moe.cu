// moe.cu -- a whole mixture-of-experts layer for a few tokens (up to 64), in two
// kernels.  With e_j, w_j a token's experts and weights and W13[e] = (gate; up):
//     y = sum_j w_j W2[e_j] h_j,   h_j = silu(gate[e_j] x) * (up[e_j] x)
// The weights are bf16 or 8 bits with a scale for each tile of 128 x 128; x, h and
// y are bf16.  h is kept as w_j h_j, rounded once to bf16, half a step of the
// output's own rounding for each of I terms of differing sign; sums are fp32.
//
// What bounds it is reading the reached experts' weights once: 3 H I elements
// each.  Both kernels read them as few_rows.cu does: a lane takes 16 bytes of a
// weight row at a time, straight to registers, and they are mma.sync's M side
// (16 weight rows), the tokens of the expert its N side, k in the order in which
// the bytes lie.
//   k_moe_up    a CTA's unit is eight features of one expert, gate and up rows
//               together: lane by lane the two stand in one accumulator, and the
//               warps, which cut k, add up through shared memory.
//   k_moe_down  a CTA owns 16 output features and all experts: the list of
//               (expert, k) is cut among its warps, so the sum over a token's
//               experts needs no atomics and no second pass, and its order is fixed.
//               It starts while k_moe_up ends, and its first weights are on the
//               way before it waits for h.
// Who has which tokens is worked out by each CTA from the T x k choices: a mask of
// tokens for each expert.  An expert chosen twice by a token counts once, with the
// sum of the weights.
#include "common.cuh"
#include "internal.h"
#include "pair.cuh"

namespace bsl {
namespace {

constexpr int kMaxTokens = BSL_MOE_MAX_TOKENS;
constexpr int kMaxPairs = kMaxTokens * BSL_ROUTE_MAX_K;
constexpr int kRows = 8;  // tokens in a group (MMA N)
static_assert(kMaxTokens <= 64, "a mask of 64 bits");

struct MoeArgs {
    const uint8_t *W13, *W2;
    const float *s13, *s2;  // 8 bits
    const __nv_bfloat16 *X;
    const int32_t *experts;
    const float *weights;
    __nv_bfloat16 *h, *Y;
    int32_t *status;
    int32_t T, k, E, H, I;
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ---------------------------------------------------------------- who has which tokens

// The reached experts, in groups of up to `most` tokens, ascending.
struct Group {
    int16_t expert, rows;
    int16_t slot;  // of the group's first token, among all (expert, token) pairs
};

struct Plan {
    Group *groups;       // [at most E + T k / most, and T k]
    uint64_t *mask;      // [E] tokens of an expert
    int16_t *start;      // [E] its first slot
    uint8_t *token;      // [T k] of a slot
    float *share;        // [T k] the sum of the token's weights for the expert
    int32_t *count;      // [1] groups

    __device__ __forceinline__ Plan(uint8_t *p, int E, int pairs)
    {
        mask = reinterpret_cast<uint64_t *>(p);
        share = reinterpret_cast<float *>(mask + E);
        count = reinterpret_cast<int32_t *>(share + pairs);
        groups = reinterpret_cast<Group *>(count + 1);
        start = reinterpret_cast<int16_t *>(groups + pairs);
        token = reinterpret_cast<uint8_t *>(start + E);
    }
    __host__ __device__ static constexpr size_t bytes(int E, int pairs) { return (10 * static_cast<size_t>(E) + 11 * static_cast<size_t>(pairs) + 4 + 15) / 16 * 16; }
};

// By the whole block; shared memory is ready for all when it returns.
__device__ __forceinline__ void make_plan(const MoeArgs &a, const Plan &p, int most)
{
    const int pairs = a.T * a.k, lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) p.mask[e] = 0;
    __syncthreads();
    bool bad = false;
    for (int i = threadIdx.x; i < pairs; i += blockDim.x) {
        const int e = static_cast<int>(load_global(reinterpret_cast<const uint32_t *>(a.experts + i)));
        if (e >= 0 && e < a.E) atomicOr(reinterpret_cast<unsigned long long *>(&p.mask[e]), 1ull << (i / a.k));
        else bad = true;
    }
    if (bad && blockIdx.x == 0) set_status(a.status, BSL_ERR_INVALID_ARG);
    __syncthreads();
    if (threadIdx.x < 32) {
        int slots = 0, groups = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane, rows = e < a.E ? __popcll(p.mask[e]) : 0, n = (rows + most - 1) / most;
            int v = rows | n << 16;  // both prefix sums at once
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, v, d);
                if (lane >= d) v += o;
            }
            const int slot = slots + (v & 0xFFFF) - rows, at = groups + (v >> 16) - n;
            if (e < a.E) p.start[e] = static_cast<int16_t>(slot);
            for (int i = 0; i < n; ++i)
                p.groups[at + i] = {static_cast<int16_t>(e), static_cast<int16_t>(min(most, rows - i * most)),
                                    static_cast<int16_t>(slot + i * most)};
            v = __shfl_sync(0xffffffffu, v, 31);
            slots += v & 0xFFFF;
            groups += v >> 16;
        }
        if (lane == 0) *p.count = groups;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < pairs; i += blockDim.x) {
        const int t = i / a.k;
        const int e = static_cast<int>(load_global(reinterpret_cast<const uint32_t *>(a.experts + i)));
        if (e < 0 || e >= a.E) continue;
        bool again = false;  // an earlier choice of this token stands for this one
        float share = 0.f;
        for (int j = t * a.k; j < (t + 1) * a.k; ++j)
            if (static_cast<int>(load_global(reinterpret_cast<const uint32_t *>(a.experts + j))) == e) {
                again |= j < i;
                share += load_float(a.weights + j);
            }
        if (again) continue;
        const int slot = p.start[e] + __popcll(p.mask[e] & ((1ull << t) - 1));
        p.token[slot] = static_cast<uint8_t>(t);
        p.share[slot] = share;
    }
    __syncthreads();
}

// ---------------------------------------------------------------- a chunk: 64 bytes of 16 weight rows

// Two e4m3 codes, in the lower half of w, to two bf16: the bits s e e e e m m m
// go to the sign and to the lowest exponent and highest mantissa bits, which is
// 2^-120 of the value, subnormal codes included, and one exact product brings it
// in.  The NaN codes come out as 480 and are looked for apart (nan_codes).
__device__ __forceinline__ uint32_t bf16_of_codes(uint32_t spread)
{
    const uint32_t v = (spread & 0x007F007Fu) * 16 | (spread * 256 & 0x80008000u);
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0x7B807B80u));
    return r;
}

// Bit 7 of a byte whose code is NaN.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return (w & 0x7F7F7F7Fu) + 0x01010101u; }

// What a lane holds of a chunk of the weight: 16 bytes of rows g and g + 8.
struct Weights {
    uint4 lo, hi;
};

// ... and of a token's vector: the elements that these bytes meet.
template <bool F8>
struct Vec {
    uint4 v[F8 ? 2 : 1];
};

template <bool F8>
__device__ __forceinline__ void multiply(float (&c)[4], const Weights &w, const Vec<F8> &x)
{
    if constexpr (!F8) {
        mma_bf16(c, w.lo.x, w.hi.x, w.lo.y, w.hi.y, x.v[0].x, x.v[0].y);
        mma_bf16(c, w.lo.z, w.hi.z, w.lo.w, w.hi.w, x.v[0].z, x.v[0].w);
    }
}

// The chunk's products, added to acc: NT groups of tokens, `groups` of them live.  8 bits: the sum of the chunk times
// the rows' scales.
template <bool F8, int NT>
__device__ __forceinline__ void add_chunk(float (&acc)[NT][4], const Weights &w, const Vec<F8> (&x)[NT], int groups, float s_lo,
                                          float s_hi, uint32_t (&nan)[2])
{
    if constexpr (F8) {
        const uint32_t lo[4] = {w.lo.x, w.lo.y, w.lo.z, w.lo.w}, hi[4] = {w.hi.x, w.hi.y, w.hi.z, w.hi.w};
        float c[NT][4] = {};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            nan[0] |= nan_codes(lo[i]);
            nan[1] |= nan_codes(hi[i]);
            const uint32_t a0 = bf16_of_codes(__byte_perm(lo[i], 0, 0x4140)), a1 = bf16_of_codes(__byte_perm(hi[i], 0, 0x4140));
            const uint32_t a2 = bf16_of_codes(__byte_perm(lo[i], 0, 0x4342)), a3 = bf16_of_codes(__byte_perm(hi[i], 0, 0x4342));
#pragma unroll
            for (int n = 0; n < NT; ++n)
                if (n < groups) {
                    const uint4 &v = x[n].v[i / 2];
                    mma_bf16(c[n], a0, a1, a2, a3, i & 1 ? v.z : v.x, i & 1 ? v.w : v.y);
                }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            acc[n][0] += s_lo * c[n][0], acc[n][1] += s_lo * c[n][1];
            acc[n][2] += s_hi * c[n][2], acc[n][3] += s_hi * c[n][3];
        }
    } else {
#pragma unroll
        for (int n = 0; n < NT; ++n)
            if (n < groups) multiply<F8>(acc[n], w, x[n]);
    }
}

// Elements of a chunk.
template <bool F8>
constexpr int chunk_of() { return F8 ? 64 : 32; }

// NaN codes in a lane's rows: to the row's other lanes (the four of a group), and into its sums.
template <int NT>
__device__ __forceinline__ void spread_nan(float (&acc)[NT][4], const uint32_t (&nan)[2])
{
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        uint32_t any = nan[r] & 0x80808080u;
        any |= __shfl_xor_sync(0xffffffffu, any, 1);
        any |= __shfl_xor_sync(0xffffffffu, any, 2);
        if (any)
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[n][2 * r] = acc[n][2 * r + 1] = __uint_as_float(0x7FC00000u);
    }
}

template <bool F8>
__device__ __forceinline__ Vec<F8> load_vec(const __nv_bfloat16 *row, int at, bool exists)
{
    Vec<F8> x;
#pragma unroll
    for (int i = 0; i < (F8 ? 2 : 1); ++i) {
        x.v[i] = make_uint4(0, 0, 0, 0);
        if (exists) x.v[i] = load_global(reinterpret_cast<const uint4 *>(row + at) + i);
    }
    return x;
}

// ---------------------------------------------------------------- gate and up

constexpr int kUpWarps = 8;

template <bool F8, int NT>
__global__ void __launch_bounds__(kUpWarps * 32, NT == 4 ? 2 : 3) k_moe_up(const MoeArgs a)
{
    // chunks of the weight on the way at once, and of the tokens' vectors (which come from L1 and L2)
    constexpr int U = NT == 4 ? 2 : 4, V = F8 ? (NT == 1 ? 2 : 1) : U, SPAN = chunk_of<F8>();
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float part[kUpWarps][NT * kRows][17];
    const Plan plan(smem, a.E, a.T * a.k);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    wait_for_prior_grid();
    // behind the wait: what came before this kernel has ended when the next one starts, which reads choices and
    // weights before its own wait
    dependents_may_launch();
    make_plan(a, plan, NT * kRows);
    const int tiles = a.I / 8, units = *plan.count * tiles;
    const int chunks = (a.H + SPAN - 1) / SPAN, kb = (a.H + 127) / 128;
    const int64_t bytes = static_cast<int64_t>(a.H) * (F8 ? 1 : 2), up_rows = a.I * bytes;

    for (int u = blockIdx.x; u < units; u += gridDim.x) {
        const Group group = plan.groups[u / tiles];
        const int live = (group.rows + kRows - 1) / kRows, i0 = u % tiles * 8;
        const uint8_t *rows = a.W13 + (static_cast<int64_t>(group.expert) * 2 * a.I + i0 + g) * bytes + 16 * t;
        const float *plane = F8 ? a.s13 + static_cast<int64_t>((2 * a.I + 127) / 128) * kb * group.expert : nullptr;
        const float *s_gate = plane + i0 / 128 * static_cast<int64_t>(kb), *s_up = plane + (a.I + i0) / 128 * static_cast<int64_t>(kb);
        const __nv_bfloat16 *x[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = 8 * n + g;
            x[n] = a.X + (r < group.rows ? static_cast<int64_t>(plan.token[group.slot + r]) * a.H : 0) + SPAN / 4 * t;
        }
        float acc[NT][4] = {};
        uint32_t nan[2] = {};
        for (int c0 = warp; c0 < chunks; c0 += kUpWarps * U) {
            Weights w[U];
            float sg[U], su[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int c = c0 + i * kUpWarps;
                w[i].lo = w[i].hi = make_uint4(0, 0, 0, 0);
                if (c * SPAN + t * (SPAN / 4) < a.H) {
                    w[i].lo = load_stream(rows + static_cast<int64_t>(c) * 64);
                    w[i].hi = load_stream(rows + up_rows + static_cast<int64_t>(c) * 64);
                }
                sg[i] = su[i] = 0.f;
                if (F8 && c < chunks) sg[i] = load_float(s_gate + c / 2), su[i] = load_float(s_up + c / 2);
            }
            Vec<F8> v[V][NT];
#pragma unroll
            for (int j = 0; j < U; j += V) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int c = c0 + (i + j) * kUpWarps;
                    const bool in = c * SPAN + t * (SPAN / 4) < a.H;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        if (n < live) v[i][n] = load_vec<F8>(x[n], c * SPAN, in && 8 * n + g < group.rows);
                }
#pragma unroll
                for (int i = 0; i < V; ++i) add_chunk<F8, NT>(acc, w[i + j], v[i], live, sg[i + j], su[i + j], nan);
            }
        }
        if (F8) spread_nan<NT>(acc, nan);
#pragma unroll
        for (int n = 0; n < NT; ++n)
            if (n < live)
#pragma unroll
                for (int i = 0; i < 4; ++i) part[warp][8 * n + 2 * t + (i & 1)][g + 8 * (i >> 1)] = acc[n][i];
        __syncthreads();
        for (int i = threadIdx.x; i < group.rows * 8; i += kUpWarps * 32) {
            const int r = i / 8, f = i % 8;
            float gate = 0.f, up = 0.f;
#pragma unroll
            for (int j = 0; j < kUpWarps; ++j) gate += part[j][r][f], up += part[j][r][f + 8];
            // (__expf is off by some 2^-20, the rounding of h by up to 2^-8)
            const float h = gate / (1.f + __expf(-gate)) * up * plan.share[group.slot + r];
            a.h[static_cast<int64_t>(group.slot + r) * a.I + i0 + f] = __float2bfloat16(h);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- down

// CTAs of a cluster share the list of a tile of 16 features, so that few tiles keep the SMs busy too.
template <int NT>
struct Down {
    static constexpr int WARPS = NT == 1 ? 16 : 8;
    static constexpr int STRIDE = 17;  // of a token's 16 sums
    static size_t bytes(int T) { return static_cast<size_t>(WARPS) * T * STRIDE * 4; }
};

template <bool F8, int NT>
__global__ void __launch_bounds__(Down<NT>::WARPS * 32, 2) k_moe_down(const MoeArgs a, const int parts)
{
    constexpr int U = 4, WARPS = Down<NT>::WARPS, STRIDE = Down<NT>::STRIDE, SPAN = chunk_of<F8>();
    extern __shared__ __align__(16) uint8_t smem[];
    const Plan plan(smem, a.E, a.T * a.k);
    float *sums = reinterpret_cast<float *>(smem + Plan::bytes(a.E, a.T * a.k));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int n0 = blockIdx.x / parts * 16, rank = blockIdx.x % parts;
    dependents_may_launch();
    for (int i = threadIdx.x; i < WARPS * a.T * STRIDE; i += WARPS * 32) sums[i] = 0.f;
    make_plan(a, plan, NT * kRows);

    const int chunks = (a.I + SPAN - 1) / SPAN, kb = (a.I + 127) / 128;
    const int64_t bytes = static_cast<int64_t>(a.I) * (F8 ? 1 : 2), nb = (a.H + 127) / 128;
    const bool in0 = n0 + g < a.H, in1 = n0 + g + 8 < a.H;
    // this warp's run of all (group, chunk) pairs
    const int64_t all = static_cast<int64_t>(*plan.count) * chunks, workers = WARPS * parts, me = rank * WARPS + warp;
    const int64_t q0 = all * me / workers;
    int left = static_cast<int>(all * (me + 1) / workers - q0);
    int at = static_cast<int>(q0 / chunks), c = static_cast<int>(q0 - static_cast<int64_t>(at) * chunks);

    // what is fetched next: group, chunk, how many are left
    int fat = at, fc = c, fleft = left;
    Weights w[U];
    float s[U];
    const uint8_t *rows = nullptr;
    const float *s2 = nullptr;
    auto open = [&] {
        const int64_t e = plan.groups[fat].expert;
        rows = a.W2 + (e * a.H + n0 + g) * bytes + 16 * t;
        if (F8) s2 = a.s2 + (e * nb + n0 / 128) * kb;
    };
    auto fetch = [&](int i) {
        if (fleft-- <= 0) return;
        const bool in = fc * SPAN + t * (SPAN / 4) < a.I;
        w[i].lo = w[i].hi = make_uint4(0, 0, 0, 0);
        if (in && in0) w[i].lo = load_stream(rows + static_cast<int64_t>(fc) * 64);
        if (in && in1) w[i].hi = load_stream(rows + 8 * bytes + static_cast<int64_t>(fc) * 64);
        if (F8) s[i] = load_float(s2 + fc / 2);
        if (++fc == chunks) {
            fc = 0, ++fat;
            if (fleft > 0) open();
        }
    };
    if (left > 0) open();
#pragma unroll
    for (int i = 0; i < U; ++i) fetch(i);
    wait_for_prior_grid();  // h is there
    float acc[NT][4] = {};
    uint32_t nan[2] = {};
    float *mine = sums + warp * a.T * STRIDE;
    while (left > 0) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (left <= 0) break;
            const Group group = plan.groups[at];
            const int live = (group.rows + kRows - 1) / kRows, k = c * SPAN + t * (SPAN / 4);
            Vec<F8> v[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n)
                if (n < live)
                    v[n] = load_vec<F8>(a.h + static_cast<int64_t>(group.slot + 8 * n + g) * a.I, k, k < a.I && 8 * n + g < group.rows);
            add_chunk<F8, NT>(acc, w[i], v, live, s[i], s[i], nan);
            fetch(i);
            --left;
            const bool last = ++c == chunks;
            if (last || left == 0) {  // the group's sum, as far as this warp has it, to its tokens
                if (F8) spread_nan<NT>(acc, nan);
                nan[0] = nan[1] = 0;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int r = 8 * n + 2 * t + (j & 1);
                        if (r < group.rows) mine[plan.token[group.slot + r] * STRIDE + g + 8 * (j >> 1)] += acc[n][j];
                        acc[n][j] = 0.f;
                    }
                __syncwarp();
            }
            if (last) c = 0, ++at;
        }
    }
    __syncthreads();
    // the warps' sums in order, then the CTAs' in order
    for (int i = threadIdx.x; i < a.T * 16; i += WARPS * 32) {
        const int r = i / 16, f = i % 16;
        float y = 0.f;
#pragma unroll
        for (int j = 0; j < WARPS; ++j) y += sums[(j * a.T + r) * STRIDE + f];
        if (parts > 1) sums[r * STRIDE + f] = y;  // (nobody else reads or writes this one)
        else if (n0 + f < a.H) a.Y[static_cast<int64_t>(r) * a.H + n0 + f] = __float2bfloat16(y);
    }
    if (parts == 1) return;
    cluster_sync_all();
    for (int i = rank * WARPS * 32 + threadIdx.x; i < a.T * 16; i += parts * WARPS * 32) {
        const int r = i / 16, f = i % 16;
        float y = 0.f;
        for (int p = 0; p < parts; ++p) {
            float other;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(other) : "r"(cluster_addr(sums + r * STRIDE + f, p)) : "memory");
            y += other;
        }
        if (n0 + f < a.H) a.Y[static_cast<int64_t>(r) * a.H + n0 + f] = __float2bfloat16(y);
    }
    cluster_sync_all();  // until the others have read this CTA's sums
}

template <bool F8, int NT>
bsl_status run(const MoeArgs &a, cudaStream_t s)
{
    const int pairs = a.T * a.k;
    const size_t plan = Plan::bytes(a.E, pairs), down = plan + Down<NT>::bytes(a.T);
    const size_t part = static_cast<size_t>(kUpWarps) * NT * kRows * 17 * 4;
    constexpr int kMost = 96 * 1024;
    if (plan + part > 48 * 1024) {
        const bsl_status sa = set_smem_once(reinterpret_cast<const void *>(&k_moe_up<F8, NT>), kMost);
        if (sa != BSL_OK) return sa;
    }
    if (down > 48 * 1024) {
        const bsl_status sa = set_smem_once(reinterpret_cast<const void *>(&k_moe_down<F8, NT>), kMost);
        if (sa != BSL_OK) return sa;
    }
    const int64_t units = static_cast<int64_t>(a.I / 8) * (pairs < a.E ? pairs : a.E);
    const int64_t room = static_cast<int64_t>(num_sms()) * (NT == 4 ? 2 : 3);
    const bsl_status up = cuda_status(launch_dependent(k_moe_up<F8, NT>, static_cast<unsigned>(units < room ? units : room),
                                                       kUpWarps * 32, plan, s, a));
    if (up != BSL_OK) return up;
    // as many CTAs a tile as two an SM have room for
    const int tiles = (a.H + 15) / 16;
    int parts = 1;
    while (parts < 8 && 2 * parts * tiles <= 2 * num_sms()) parts *= 2;
    return cuda_status(launch_dependent_cluster(k_moe_down<F8, NT>, tiles * parts, parts, Down<NT>::WARPS * 32, down, s, a, parts));
}

// Tokens a group takes: as many as an expert has on the average, in eights.  An expert with more is read again for
// its next group, mostly from L2, by CTAs that run at about the same time.
template <bool F8>
bsl_status run(const MoeArgs &a, cudaStream_t s)
{
    const int reach = a.T * a.k, mean = (reach + a.E - 1) / a.E;
    const int rows = a.T < mean ? a.T : mean;
    return rows <= kRows ? run<F8, 1>(a, s) : rows <= 2 * kRows ? run<F8, 2>(a, s) : run<F8, 4>(a, s);
}

}  // namespace

bsl_status launch_moe(const void *X, int32_t T, const int32_t *experts, const float *weights, int32_t k, const void *W13,
                      const float *s13, const void *W2, const float *s2, int32_t E, int32_t H, int32_t I, int32_t *status,
                      void *workspace, void *Y, cudaStream_t s)
{
    MoeArgs a = {};
    a.W13 = static_cast<const uint8_t *>(W13);
    a.W2 = static_cast<const uint8_t *>(W2);
    a.s13 = s13;
    a.s2 = s2;
    a.X = static_cast<const __nv_bfloat16 *>(X);
    a.experts = experts;
    a.weights = weights;
    a.h = static_cast<__nv_bfloat16 *>(workspace);
    a.Y = static_cast<__nv_bfloat16 *>(Y);
    a.status = status;
    a.T = T;
    a.k = k;
    a.E = E;
    a.H = H;
    a.I = I;
    return s13 ? run<true>(a, s) : run<false>(a, s);
}

}  // namespace bsl
