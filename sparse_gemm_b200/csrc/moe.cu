// moe.cu -- a whole mixture-of-experts layer for a few tokens (up to 64), in two
// kernels.  With e_j, w_j a token's experts and weights and W13[e] = (gate; up):
//     y = sum_j w_j W2[e_j] h_j,   h_j = silu(gate[e_j] x) * (up[e_j] x)
// The weights are bf16 or 8 bits with a scale for each tile of 128 x 128; x, h and
// y are bf16.  h is kept as w_j h_j, rounded once to bf16, half a step of the
// output's own rounding for each of I terms of differing sign; sums are fp32.
//
// What bounds it is reading the reached experts' weights once: 3 H I elements
// each.  Both kernels bring them through a ring of asynchronous copies a warp
// (ring.cuh), and they are mma.sync's M side (16 weight rows), the tokens of the
// expert its N side, k in the order in which the bytes lie; 8-bit weights become bf16
// by bit moves, exactly.  Measured: one token, two experts of 4096 x 14336 in bf16, up 75 us
// (6.2 TB/s), down 42 (5.6); 32 tokens, 64 experts of 2048 x 1408 in 8 bits, up 105, down 63,
// which instructions bound (442 for a step of 2 KB, the issue slots 69 % used), not the
// bytes (85 for both).  With the weights loaded straight to registers: 75, 52, 137, 79.
//   k_moe_up    a CTA's unit is eight features of one expert, gate and up rows
//               together: lane by lane the two stand in one accumulator, and the
//               warps, which cut k, add up through shared memory.
//   k_moe_down  a CTA, or a cluster where such tiles are few, owns 16 output features
//               and all experts: the list of (expert, k) is cut among its warps, so the
//               sum over a token's experts needs no atomics and no second pass, and its
//               order is fixed.
//               It starts while k_moe_up ends, and its first weights are on the
//               way before it waits for h.
// Who has which tokens is worked out by each CTA from the T x k choices: a mask of
// tokens for each expert.  An expert chosen twice by a token counts once, with the
// sum of the weights.
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "pair.cuh"
#include "ring.cuh"

namespace bsl {
namespace {

constexpr int kMaxTokens = BSL_MOE_MAX_TOKENS;
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

// ---------------------------------------------------------------- steps: 64 bf16 elements, or a block of 128 codes

template <bool F8>
constexpr int step_of() { return F8 ? 128 : 64; }  // elements

// What the lane's bytes of a step meet of a token's vector.
template <bool F8>
struct Vec {
    uint4 v[F8 ? 4 : 2];  // of unit t, and of unit 4 + t
};

template <bool F8>
__device__ __forceinline__ void load_vec(Vec<F8> &x, const __nv_bfloat16 *row, int k0, int t, int K, bool exists)
{
    constexpr int UNIT = F8 ? 16 : 8;  // elements
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int k = k0 + (4 * h + t) * UNIT;
        const bool in = exists && k < K;
#pragma unroll
        for (int i = 0; i < UNIT / 8; ++i) {
            uint4 &v = x.v[h * (UNIT / 8) + i];
            v = make_uint4(0, 0, 0, 0);
            if (in) v = load_global(reinterpret_cast<const uint4 *>(row + k) + i);
        }
    }
}

// Four e4m3 codes to two registers of two bf16, codes 0, 2 and codes 1, 3: the bits s e e e e m m m go to the sign and
// to the lowest exponent and highest mantissa bits, which is 2^-120 of the value, subnormal codes included, and one
// exact product brings it to 2^-9 of the value, 0.875 at most: a block's sum over tokens of up to 10^36 stays finite.  The
// sums of all blocks get the 2^9 back at the end (code_unit; in the scales it took 177 us for 171: 32 tokens, six of 64
// experts of 2048 x 1408).  The NaN codes come out as 480 and are looked for apart: they, and no other, have bit 7
// of their byte set in what is returned.
__device__ __forceinline__ uint32_t decode4(uint32_t w, uint32_t &even, uint32_t &odd)
{
    const uint32_t m = w & 0x7F7F7F7Fu;
    even = (w * 256 & 0x80008000u) | (m & 0x007F007Fu) * 16;
    odd = (w & 0x80008000u) | (m >> 4 & 0x07F007F0u);
    asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(even) : "r"(0x77007700u));
    asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(odd) : "r"(0x77007700u));
    return m + 0x01010101u;
}

template <bool F8>
constexpr float code_unit() { return F8 ? 512.f : 1.f; }

// A step's products, added to acc: NT groups of tokens, `live` of them there.  8 bits: the sum of the block times the
// rows' scales; the codes of a word are taken as 0, 2 and 1, 3, and so are the tokens' elements.
template <bool F8, int NT>
__device__ __forceinline__ void add_step(float (&acc)[NT][4], const uint8_t *slot, const Vec<F8> (&x)[NT], int live, float s_lo,
                                         float s_hi, uint32_t (&nan)[2])
{
    float c[NT][4] = {};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint4 wl, wh;
        read_step(slot, h, wl, wh);
        if constexpr (F8) {
            const uint32_t lo[4] = {wl.x, wl.y, wl.z, wl.w}, hi[4] = {wh.x, wh.y, wh.z, wh.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t a[4];
                nan[0] |= decode4(lo[i], a[0], a[2]);
                nan[1] |= decode4(hi[i], a[1], a[3]);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    if (n < live) {
                        const uint4 &v = x[n].v[2 * h + i / 2];
                        const uint32_t b0 = i & 1 ? v.z : v.x, b1 = i & 1 ? v.w : v.y;
                        mma_bf16(c[n], a[0], a[1], a[2], a[3], __byte_perm(b0, b1, 0x5410), __byte_perm(b0, b1, 0x7632));
                    }
            }
        } else {
#pragma unroll
            for (int n = 0; n < NT; ++n)
                if (n < live) {
                    const uint4 &v = x[n].v[h];
                    mma_bf16(acc[n], wl.x, wh.x, wl.y, wh.y, v.x, v.y);
                    mma_bf16(acc[n], wl.z, wh.z, wl.w, wh.w, v.z, v.w);
                }
        }
    }
    if constexpr (F8) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            acc[n][0] += s_lo * c[n][0], acc[n][1] += s_lo * c[n][1];
            acc[n][2] += s_hi * c[n][2], acc[n][3] += s_hi * c[n][3];
        }
    }
}

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

// CTAs of an SM that the kernels are compiled for.
constexpr int ctas_of(int NT) { return NT == 1 ? 3 : 2; }

constexpr size_t ring_bytes(int ring) { return static_cast<size_t>(kWarps) * ring * kStep; }

// ---------------------------------------------------------------- gate and up

constexpr int kUpRing = 4;

template <bool F8, int NT>
__global__ void __launch_bounds__(kWarps * 32, ctas_of(NT)) k_moe_up(const MoeArgs a, const int team)
{
    constexpr int SPAN = step_of<F8>();
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float part[kWarps][NT * kRows][17];
    const Plan plan(smem + ring_bytes(kUpRing), a.E, a.T * a.k);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    uint8_t *ring = smem + warp * kUpRing * kStep;
    const int mine = warp / team, member = warp % team, teams = kWarps / team, stride = gridDim.x * teams;
    wait_for_prior_grid();
    // behind the wait: what came before this kernel has ended when the next one starts, which reads choices and
    // weights before its own wait
    dependents_may_launch();
    make_plan(a, plan, NT * kRows);
    const int tiles = a.I / 8, units = *plan.count * tiles;
    const int steps = (a.H + SPAN - 1) / SPAN, kb = (a.H + 127) / 128;
    const int64_t bytes = static_cast<int64_t>(a.H) * (F8 ? 1 : 2), up_rows = a.I * bytes;
    const int64_t off[4] = {0, 4 * bytes, up_rows, up_rows + 4 * bytes};

    // the copies' place: unit of work, step, and the lane's first byte there
    int fu = member < steps ? blockIdx.x * teams + mine : units, fc = member, slot = 0;
    const uint8_t *from = nullptr;
    auto open = [&] {
        if (fu < units)
            from = a.W13 + (static_cast<int64_t>(plan.groups[fu / tiles].expert) * 2 * a.I + fu % tiles * 8 + (lane >> 3)) * bytes +
                   16 * (lane & 7);
    };
    auto issue = [&](int at) {
        if (fu < units) {
            const int64_t first = static_cast<int64_t>(fc) * 128;
            const bool in = first + 16 * (lane & 7) < bytes, exists[4] = {in, in, in, in};
            copy_step(ring + at * kStep, from + first, off, exists, a.W13);
            if ((fc += team) >= steps) {
                fc = member;
                fu += stride;
                open();
            }
        }
        copies_commit();
    };
    open();
#pragma unroll
    for (int i = 0; i < kUpRing; ++i) issue(i);
    for (int u = blockIdx.x * teams + mine; u < units; u += stride) {
        const Group group = plan.groups[u / tiles];
        const int live = (group.rows + kRows - 1) / kRows, i0 = u % tiles * 8;
        const float *plane = F8 ? a.s13 + static_cast<int64_t>((2 * a.I + 127) / 128) * kb * group.expert : nullptr;
        const float *s_gate = plane + i0 / 128 * static_cast<int64_t>(kb), *s_up = plane + (a.I + i0) / 128 * static_cast<int64_t>(kb);
        const __nv_bfloat16 *x[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = 8 * n + g;
            x[n] = a.X + (r < group.rows ? static_cast<int64_t>(plan.token[group.slot + r]) * a.H : 0);
        }
        float acc[NT][4] = {};
        uint32_t nan[2] = {};
        for (int c = member; c < steps; c += team) {
            Vec<F8> v[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n)
                if (n < live) load_vec<F8>(v[n], x[n], c * SPAN, t, a.H, 8 * n + g < group.rows);
            const float sg = F8 ? load_float(s_gate + c) : 1.f, su = F8 ? load_float(s_up + c) : 1.f;
            copies_wait<kUpRing>();
            add_step<F8, NT>(acc, ring + slot * kStep, v, live, sg, su, nan);
            __syncwarp();
            issue(slot);
            slot = (slot + 1) % kUpRing;
        }
        if (F8) spread_nan<NT>(acc, nan);
#pragma unroll
        for (int n = 0; n < NT; ++n)
            if (n < live)
#pragma unroll
                for (int i = 0; i < 4; ++i) part[warp][8 * n + 2 * t + (i & 1)][g + 8 * (i >> 1)] = acc[n][i];
        named_bar_sync(1 + mine, 32 * team);
        for (int i = threadIdx.x - 32 * team * mine; i < group.rows * 8; i += 32 * team) {
            const int r = i / 8, f = i % 8;
            float gate = 0.f, up = 0.f;
            for (int j = mine * team; j < (mine + 1) * team; ++j) gate += part[j][r][f], up += part[j][r][f + 8];  // in order
            gate *= code_unit<F8>(), up *= code_unit<F8>();
            // (__expf is off by 2 + 1.2 |gate| units of 2^-23, 2^-16 where it last matters; the rounding of h by up to 2^-8)
            const float h = gate / (1.f + __expf(-gate)) * up * plan.share[group.slot + r];
            a.h[static_cast<int64_t>(group.slot + r) * a.I + i0 + f] = __float2bfloat16(h);
        }
        named_bar_sync(1 + mine, 32 * team);
    }
    copies_end();
}

// ---------------------------------------------------------------- down

constexpr int kStride = 17;   // of a token's 16 sums

size_t sums_bytes(int T) { return static_cast<size_t>(kWarps) * T * kStride * 4; }

// CTAs of an SM, and steps under way in each warp: more CTAs with shorter rings where the registers are few (one token,
// two experts of 4096 x 14336 in bf16, the whole call: 136 us with four CTAs and three steps, 144 with three CTAs and four
// steps, 147 with two and four).  The 8-bit kernel spills with more than two (32 tokens: 171 us, 200 with three CTAs).
constexpr bool light(bool f8, int NT) { return !f8 && NT == 1; }
constexpr int down_ctas(bool f8, int NT) { return light(f8, NT) ? 4 : 2; }
constexpr int down_ring(bool f8, int NT) { return light(f8, NT) ? 3 : 4; }

// CTAs of a cluster share the list of a tile of 16 features, so that few tiles keep the SMs busy too.
template <bool F8, int NT>
__global__ void __launch_bounds__(kWarps * 32, down_ctas(F8, NT)) k_moe_down(const MoeArgs a, const int parts)
{
    constexpr int SPAN = step_of<F8>(), RING = down_ring(F8, NT);
    extern __shared__ __align__(16) uint8_t smem[];
    const Plan plan(smem + ring_bytes(RING), a.E, a.T * a.k);
    float *sums = reinterpret_cast<float *>(smem + ring_bytes(RING) + Plan::bytes(a.E, a.T * a.k));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    uint8_t *ring = smem + warp * RING * kStep;
    const int n0 = blockIdx.x / parts * 16, rank = blockIdx.x % parts;
    dependents_may_launch();
    for (int i = threadIdx.x; i < kWarps * a.T * kStride; i += kWarps * 32) sums[i] = 0.f;
    make_plan(a, plan, NT * kRows);

    const int steps = (a.I + SPAN - 1) / SPAN, kb = (a.I + 127) / 128;
    const int64_t bytes = static_cast<int64_t>(a.I) * (F8 ? 1 : 2), nb = (a.H + 127) / 128;
    const int64_t off[4] = {0, 4 * bytes, 8 * bytes, 12 * bytes};
    // This warp's share of all (group, step) pairs: every so many steps of each group, so that the warps read side by
    // side (one token, two experts of 4096 x 14336 in bf16, then with two CTAs an SM: 54 us, runs 56); or, where that is not some steps a group,
    // a run of the whole list.
    const int workers = kWarps * parts, me = rank * kWarps + warp;
    const int64_t all = static_cast<int64_t>(*plan.count) * steps, q0 = all * me / workers;
    int slot = 0, at = 0, c = me, begin = me, inc = workers;
    int left = *plan.count * ((steps - me + workers - 1) / workers);
    if (steps < 4 * workers) {
        left = static_cast<int>(all * (me + 1) / workers - q0);
        at = static_cast<int>(q0 / steps);
        c = static_cast<int>(q0 - static_cast<int64_t>(at) * steps);
        begin = 0;
        inc = 1;
    }

    // the copies' place: group, step, how many are left
    int fat = at, fc = c, fleft = left;
    const uint8_t *from = nullptr;
    auto open = [&] {
        if (fleft > 0)
            from = a.W2 + (static_cast<int64_t>(plan.groups[fat].expert) * a.H + n0 + (lane >> 3)) * bytes + 16 * (lane & 7);
    };
    auto issue = [&](int into) {
        if (fleft > 0) {
            const int64_t first = static_cast<int64_t>(fc) * 128;
            const bool in = first + 16 * (lane & 7) < bytes;
            const int rows = a.H - n0 - (lane >> 3);
            const bool exists[4] = {in && rows > 0, in && rows > 4, in && rows > 8, in && rows > 12};
            copy_step(ring + into * kStep, from + first, off, exists, a.W2);
            --fleft;
            if ((fc += inc) >= steps) {
                fc = begin;
                ++fat;
                open();
            }
        }
        copies_commit();
    };
    open();
#pragma unroll
    for (int i = 0; i < RING; ++i) issue(i);
    wait_for_prior_grid();  // h is there
    // h comes from L2 (every CTA reads all of it), so the loads are P steps ahead where registers allow it
    constexpr int P = F8 && NT > 1 || NT > 2 ? 1 : 2;
    Vec<F8> v[P][NT];
    float s[P];
    int vat = at, vc = c, vleft = left;
    auto load = [&](int i) {
        if (vleft <= 0) return;
        const Group group = plan.groups[vat];
#pragma unroll
        for (int n = 0; n < NT; ++n)
            if (8 * n < group.rows)
                load_vec<F8>(v[i][n], a.h + static_cast<int64_t>(group.slot + 8 * n + g) * a.I, vc * SPAN, t, a.I, 8 * n + g < group.rows);
        s[i] = F8 ? load_float(a.s2 + (group.expert * nb + n0 / 128) * kb + vc) : 1.f;
        --vleft;
        if ((vc += inc) >= steps) {
            vc = begin;
            ++vat;
        }
    };
#pragma unroll
    for (int i = 0; i < P; ++i) load(i);
    float acc[NT][4] = {};
    uint32_t nan[2] = {};
    float *mine = sums + warp * a.T * kStride;
    while (left > 0) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            if (left <= 0) break;
            const Group group = plan.groups[at];
            copies_wait<RING>();
            add_step<F8, NT>(acc, ring + slot * kStep, v[i], (group.rows + kRows - 1) / kRows, s[i], s[i], nan);
            __syncwarp();
            issue(slot);
            load(i);
            slot = (slot + 1) % RING;
            const bool last = (c += inc) >= steps;
            if (last || left == 1) {  // the group's sum, as far as this warp has it, to its tokens
                if (F8) spread_nan<NT>(acc, nan);
                nan[0] = nan[1] = 0;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int r = 8 * n + 2 * t + (j & 1);
                        if (r < group.rows) mine[plan.token[group.slot + r] * kStride + g + 8 * (j >> 1)] += acc[n][j];
                        acc[n][j] = 0.f;
                    }
                __syncwarp();
            }
            if (last) c = begin, ++at;
            --left;
        }
    }
    copies_end();
    __syncthreads();
    // the warps' sums in order, then the CTAs' in order
    for (int i = threadIdx.x; i < a.T * 16; i += kWarps * 32) {
        const int r = i / 16, f = i % 16;
        float y = 0.f;
#pragma unroll
        for (int j = 0; j < kWarps; ++j) y += sums[(j * a.T + r) * kStride + f];
        if (parts > 1) sums[r * kStride + f] = y;  // (nobody else reads or writes this one)
        else if (n0 + f < a.H) a.Y[static_cast<int64_t>(r) * a.H + n0 + f] = __float2bfloat16(y * code_unit<F8>());
    }
    if (parts == 1) return;
    cluster_sync_all();
    for (int i = rank * kWarps * 32 + threadIdx.x; i < a.T * 16; i += parts * kWarps * 32) {
        const int r = i / 16, f = i % 16;
        float y = 0.f;
        for (int p = 0; p < parts; ++p) {
            float other;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(other) : "r"(cluster_addr(sums + r * kStride + f, p)) : "memory");
            y += other;
        }
        if (n0 + f < a.H) a.Y[static_cast<int64_t>(r) * a.H + n0 + f] = __float2bfloat16(y * code_unit<F8>());
    }
    cluster_sync_all();  // until the others have read this CTA's sums
}

template <bool F8, int NT>
bsl_status run(const MoeArgs &a, cudaStream_t s)
{
    constexpr int kMost = 150 * 1024;
    const int pairs = a.T * a.k;
    const size_t plan = Plan::bytes(a.E, pairs), up = ring_bytes(kUpRing) + plan;
    const size_t down = ring_bytes(down_ring(F8, NT)) + plan + sums_bytes(a.T);
    bsl_status st = set_smem_once(reinterpret_cast<const void *>(&k_moe_up<F8, NT>), kMost);
    if (st == BSL_OK) st = set_smem_once(reinterpret_cast<const void *>(&k_moe_down<F8, NT>), kMost);
    if (st != BSL_OK) return st;
    const int64_t units = static_cast<int64_t>(a.I / 8) * (pairs < a.E ? pairs : a.E);
    const int64_t room = static_cast<int64_t>(num_sms()) * ctas_of(NT);
    const int team = team_of((a.H + step_of<F8>() - 1) / step_of<F8>());
    const int64_t ctas = (units * team + kWarps - 1) / kWarps;
    st = cuda_status(launch_dependent(k_moe_up<F8, NT>, static_cast<unsigned>(ctas < room ? ctas : room), kWarps * 32, up, s, a, team));
    if (st != BSL_OK) return st;
    // as many CTAs a tile as there is room for
    const int tiles = (a.H + 15) / 16;
    int parts = 1;
    const int fit = static_cast<int>(227 * 1024 / (down + 1024)), ctas_an_sm = fit < down_ctas(F8, NT) ? fit : down_ctas(F8, NT);
    while (parts < 8 && 2 * parts * tiles <= ctas_an_sm * num_sms()) parts *= 2;
    return cuda_status(launch_dependent_cluster(k_moe_down<F8, NT>, tiles * parts, parts, kWarps * 32, down, s, a, parts));
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
