// few_rows.cu -- forward of the expert (grouped) layer and of the 4- and 8-bit layers for
// a few rows in all (single tokens, up to 32): Y[t] = X[t] . W[e]^T + bias[e].
//
// Each weight row that is used is read once and little else matters: bytes,
// instructions (4 bits) and latency bound it.  A block owns 16 features of one
// expert and its 8 warps cut K, so that a call spreads over every SM at once,
// with no set-up before the first load but finding the block's expert.  The
// features are mma.sync's M side, the rows of X its N side; the order of k
// inside a product is free as long as both operands share it.  The warps' fp32
// sums are added in order through shared memory, and rounded once.
#include "common.cuh"
#include "grouped.cuh"
#include "internal.h"

namespace bsl {
namespace {

constexpr int kWarps = 8;
constexpr int kRows = 8;       // rows of X in a group (MMA N); a call has up to four groups
constexpr int kFeatures = 16;  // per block (MMA M)

struct FewArgs {
    const uint8_t *W, *w_scales, *X, *x_scales;
    const __nv_bfloat16 *bias;
    __nv_bfloat16 *Y;
    const int32_t *offsets;  // null: one expert owns all rows
    int32_t *status;
    int32_t T, E, N, K, blocks;  // blocks: of one expert
    int32_t zero_rest;
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

// The li-th expert with rows, found by every warp on its own: e < 0 if there are
// not that many.  Offsets are made safe as by clamp_offsets.
struct Found {
    int e, first, rows;
};

__device__ __forceinline__ Found find_expert(const FewArgs &a, int li, int &rest_front, int &rest_back, bool &bad)
{
    Found f = {-1, 0, 0};
    bad = false;
    if (!a.offsets) {
        rest_front = 0;
        rest_back = a.T;
        if (li == 0) f = {0, 0, a.T};
        return f;
    }
    const int lane = threadIdx.x & 31;
    auto clamp = [&](int v) { return v < 0 ? 0 : v > a.T ? a.T : v; };
    const int raw0 = load_global(a.offsets);
    int carry = clamp(raw0), seen = 0;
    bad = carry != raw0;
    rest_front = carry;
    for (int i0 = 0; i0 < a.E; i0 += 32) {
        const int i = i0 + lane;
        const int raw = i < a.E ? load_global(a.offsets + i + 1) : 0;
        int v = clamp(raw);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, v, d);
            if (lane >= d && o > v) v = o;
        }
        if (v < carry) v = carry;
        bad |= i < a.E && v != raw;
        const int up = __shfl_up_sync(0xffffffffu, v, 1), prev = lane ? up : carry;
        const uint32_t live = __ballot_sync(0xffffffffu, i < a.E && v > prev);
        const int n = __popc(live);
        if (f.e < 0 && li < seen + n) {
            const int bit = __fns(live, 0, li - seen + 1);
            f.e = i0 + bit;
            f.first = __shfl_sync(0xffffffffu, prev, bit);
            f.rows = __shfl_sync(0xffffffffu, v, bit) - f.first;
        }
        seen += n;
        carry = __shfl_sync(0xffffffffu, v, 31);
    }
    rest_back = carry;
    bad = __any_sync(0xffffffffu, bad);
    return f;
}

// Zeros for the rows of no expert, in the block's features.
__device__ __forceinline__ void zero_rest_rows(const FewArgs &a, int n0, int front, int back)
{
    const int n = n0 + threadIdx.x % kFeatures;
    for (int r = threadIdx.x / kFeatures; r < a.T; r += kWarps * 32 / kFeatures)
        if ((r < front || r >= back) && n < a.N) a.Y[static_cast<int64_t>(r) * a.N + n] = __float2bfloat16(0.f);
}

// The warps' sums, in order, and the bias to the block's features of Y.
template <int NT>
__device__ __forceinline__ void add_parts(const FewArgs &a, const Found &f, int n0, const float (*part)[NT * kRows][kFeatures])
{
    const int n = n0 + threadIdx.x % kFeatures;
    if (n >= a.N) return;
    for (int r = threadIdx.x / kFeatures; r < f.rows; r += kWarps * 32 / kFeatures) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += part[w][r][threadIdx.x % kFeatures];
        if (a.bias) s += __bfloat162float(a.bias[static_cast<int64_t>(f.e) * a.N + n]);
        a.Y[static_cast<int64_t>(f.first + r) * a.N + n] = __float2bfloat16(s);
    }
}

// ---------------------------------------------------------------- bf16

// A lane reads 16 bytes of a weight row at a time, two or four steps at once, and
// feeds them to the MMA as they lie.  NT groups of eight rows: 1, 2 or 4.
template <int NT>
__global__ void __launch_bounds__(kWarps * 32, 3) k_few_rows(const FewArgs a)
{
    __shared__ float part[kWarps][NT * kRows][kFeatures];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int li = blockIdx.x / a.blocks, n0 = (blockIdx.x - li * a.blocks) * kFeatures;
    dependents_may_launch();
    wait_for_prior_grid();
    int front, back;
    bool bad;
    const Found f = find_expert(a, li, front, back, bad);
    if (bad && blockIdx.x == 0 && threadIdx.x == 0) set_status(a.status, BSL_ERR_INVALID_ARG);
    if (a.zero_rest && li == 0) zero_rest_rows(a, n0, front, back);
    if (f.e < 0) return;

    // this lane's rows: features n0 + g and n0 + g + 8 of the weight, rows g, g + 8, ... of X
    constexpr int SPAN = 32;  // k of a step: 16 bytes a lane
    const int64_t bytes = static_cast<int64_t>(a.K) * 2;
    const int64_t wr = static_cast<int64_t>(f.e) * a.N + n0 + g;
    const bool in0 = n0 + g < a.N, in1 = n0 + g + 8 < a.N;
    const uint8_t *w0 = a.W + wr * bytes + 16 * t, *w1 = w0 + 8 * bytes;
    const uint8_t *x = a.X + static_cast<int64_t>(f.first + g) * bytes + 16 * t;
    const int steps = (a.K + SPAN - 1) / SPAN;
    constexpr int U = NT == 4 ? 2 : 4;
    float acc[NT][4] = {};
    for (int s0 = warp; s0 < steps; s0 += kWarps * U) {
        uint4 va[U], vb[U], vx[U][NT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = s0 + u * kWarps;
            const bool in = s * SPAN + t * (SPAN / 4) < a.K;
            va[u] = vb[u] = make_uint4(0, 0, 0, 0);
            if (in && in0) va[u] = load_stream(w0 + static_cast<int64_t>(s) * 64);
            if (in && in1) vb[u] = load_stream(w1 + static_cast<int64_t>(s) * 64);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                vx[u][n] = make_uint4(0, 0, 0, 0);
                if (in && g + 8 * n < f.rows)
                    vx[u][n] = load_global(reinterpret_cast<const uint4 *>(x + n * 8 * bytes + static_cast<int64_t>(s) * 64));
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                mma_bf16(acc[n], va[u].x, vb[u].x, va[u].y, vb[u].y, vx[u][n].x, vx[u][n].y);
                mma_bf16(acc[n], va[u].z, vb[u].z, va[u].w, vb[u].w, vx[u][n].z, vx[u][n].w);
            }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[warp][8 * n + 2 * t + (i & 1)][g + 8 * (i >> 1)] = acc[n][i];
    __syncthreads();
    add_parts<NT>(a, f, n0, part);
}

// ---------------------------------------------------------------- 4 bits

__device__ __forceinline__ void copy16(uint8_t *dst, const uint8_t *src, bool exists)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(exists ? 16 : 0)
                 : "memory");
}

__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Eight codes to four registers of two f16, 2^-14 of their values: the bits
// s e e m at the sign and the lowest exponent and highest mantissa bits of the
// upper byte, zero and 0.5 (which f16 has as a subnormal number) included; the
// lower byte is zero.
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t (&v)[4])
{
    const uint32_t even = (w << 4 & 0x80808080u) | (w << 1 & 0x0E0E0E0Eu);
    const uint32_t odd = (w & 0x80808080u) | (w >> 3 & 0x0E0E0E0Eu);
    v[0] = even & 0xFF00FF00u;
    v[1] = __byte_perm(even, 0, 0x2404);
    v[2] = odd & 0xFF00FF00u;
    v[3] = __byte_perm(odd, 0, 0x2404);
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1, const float (&d)[4])
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %11, %12, %13};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(d[0]), "f"(d[1]), "f"(d[2]), "f"(d[3]));
}

// 2^h, -127 <= h <= 127.
__device__ __forceinline__ float power_of_2(int h) { return __uint_as_float(h > -127 ? (h + 127) << 23 : 0x400000); }

// A block's sum p (2^-28 of it) under scale bytes a and b, whatever they are.
__device__ __forceinline__ float scaled(float p, int a, int b)
{
    if (a == 255 || b == 255) return __uint_as_float(0x7FC00000u);
    const int e = a + b - 254, h = e >> 1;
    return 268435456.f * p * power_of_2(h) * power_of_2(e - h);
}

// The 32 elements of one block are an MMA's k, so its scales come in by one
// product per result, and the codes stand for themselves.  A warp's steps of
// 128 k (64 bytes of a row) come through a ring in shared memory, which also
// brings the words of a block to the lanes that hold its k.  Instructions bound
// it, 11 for eight codes and as many again for scales, loops and addresses:
// 4096 x 4096 takes 9.3 us for one row (with a bf16 product for each pair of codes to
// bring the scale in, straight from registers: 10.8), 11008 x 4096 14.2 (15.8).
// Three or four steps in flight cost blocks an SM and are no faster (9.4, 9.7),
// 32 features a block 13.3, e4m3 operands (one word for four codes) 9.7.
template <int NT>
struct Few4 {
    static constexpr int ST = 2;                          // steps in flight, a warp
    static constexpr int ROWS = kFeatures + kRows * NT;
    static constexpr int STEP = ROWS * 64;
    static constexpr int SMEM = kWarps * ST * STEP;
    static_assert(kWarps * NT * kRows * kFeatures * 4 <= SMEM, "the warps' sums take the ring's place");
};

template <int NT>
__global__ void __launch_bounds__(kWarps * 32) k_few_rows4(const FewArgs a)
{
    using C = Few4<NT>;
    constexpr int ST = C::ST;
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int li = blockIdx.x / a.blocks, n0 = (blockIdx.x - li * a.blocks) * kFeatures;
    dependents_may_launch();
    wait_for_prior_grid();
    int front, back;
    bool bad;
    const Found f = find_expert(a, li, front, back, bad);
    if (bad && blockIdx.x == 0 && threadIdx.x == 0) set_status(a.status, BSL_ERR_INVALID_ARG);
    if (a.zero_rest && li == 0) zero_rest_rows(a, n0, front, back);
    if (f.e < 0) return;

    const int blocks = a.K / 32, count = (blocks + 3) / 4, mine = (count - warp + kWarps - 1) / kWarps;
    const int64_t bytes = a.K / 2, wr = static_cast<int64_t>(f.e) * a.N + n0;
    uint8_t *ring = smem + warp * ST * C::STEP;
    // a lane copies chunk t (block t) of rows g, g + 8, ..., of the weight and then of X, and reads their scales
    const uint8_t *w = a.W + (wr + g) * bytes + 16 * t, *x = a.X + static_cast<int64_t>(f.first + g) * bytes + 16 * t;
    const uint8_t *ws = a.w_scales + (wr + g) * blocks + t, *xs = a.x_scales + static_cast<int64_t>(f.first + g) * blocks + t;
    // chunks of a row trade places by its number, so that eight rows' words of one chunk lie in different banks
    const int put = g * 64 + ((t + (g >> 1)) & 3) * 16;
    int sw[ST][2], sx[ST][NT];
    auto issue = [&](int j, int slot, int (&vw)[2], int (&vx)[NT]) {
        if (j < mine) {
            const int s = warp + j * kWarps;
            const bool in = 4 * s + t < blocks;
            uint8_t *dst = ring + slot * C::STEP + put;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const bool exists = in && n0 + g + 8 * m < a.N;
                copy16(dst + m * 512, exists ? w + m * 8 * bytes + static_cast<int64_t>(s) * 64 : a.W, exists);
                vw[m] = 127;  // (zeros under a scale of one)
                if (exists) vw[m] = load_global(ws + m * 8 * static_cast<int64_t>(blocks) + 4 * s);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const bool exists = in && g + 8 * n < f.rows;
                copy16(dst + (2 + n) * 512, exists ? x + n * 8 * bytes + static_cast<int64_t>(s) * 64 : a.X, exists);
                vx[n] = 127;
                if (exists) vx[n] = load_global(xs + n * 8 * static_cast<int64_t>(blocks) + 4 * s);
            }
        }
        copies_commit();
    };
#pragma unroll
    for (int u = 0; u < ST; ++u) issue(u, u, sw[u], sx[u]);
    float acc[NT][4] = {};
    for (int j0 = 0; j0 < mine; j0 += ST) {
#pragma unroll
        for (int u = 0; u < ST; ++u) {
            if (j0 + u >= mine) break;
            copies_wait<ST - 1>();
            __syncwarp();
            const uint8_t *src = ring + u * C::STEP + g * 64 + 4 * t;
            // scales whose products, 2^28 and all, are normal numbers: one product a result
            bool in_range = true;
#pragma unroll
            for (int m = 0; m < 2; ++m) in_range &= static_cast<uint32_t>(sw[u][m] - 50) <= 126u;
#pragma unroll
            for (int n = 0; n < NT; ++n) in_range &= static_cast<uint32_t>(sx[u][n] - 50) <= 126u;
            const bool plain = __all_sync(0xffffffffu, in_range);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int chunk = ((b + (g >> 1)) & 3) * 16;
                uint32_t r[NT][4];
                int fx[NT][2];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    codes_to_f16(*reinterpret_cast<const uint32_t *>(src + chunk + (2 + n) * 512), r[n]);
                    fx[n][0] = __shfl_sync(0xffffffffu, sx[u][n] << 23, 8 * t + b);
                    fx[n][1] = __shfl_sync(0xffffffffu, sx[u][n] << 23, 8 * t + 4 + b);
                }
                uint32_t p[4], q[4];
                codes_to_f16(*reinterpret_cast<const uint32_t *>(src + chunk), p);
                codes_to_f16(*reinterpret_cast<const uint32_t *>(src + chunk + 512), q);
                const int fw0 = __shfl_sync(0xffffffffu, sw[u][0] << 23, b, 4);
                const int fw1 = __shfl_sync(0xffffffffu, sw[u][1] << 23, b, 4);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float zero[4] = {};
                    float c[4];
                    mma_f16(c, p[0], q[0], p[1], q[1], r[n][0], r[n][1], zero);
                    mma_f16(c, p[2], q[2], p[3], q[3], r[n][2], r[n][3], c);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int s0 = i < 2 ? fw0 : fw1, s1 = fx[n][i & 1];
                        if (plain)
                            acc[n][i] += c[i] * __uint_as_float(static_cast<uint32_t>(s0) + static_cast<uint32_t>(s1) - (99u << 23));
                        else
                            acc[n][i] += scaled(c[i], s0 >> 23, s1 >> 23);
                    }
                }
            }
            __syncwarp();
            issue(j0 + u + ST, u, sw[u], sx[u]);
        }
    }
    copies_wait<0>();
    __syncthreads();
    auto part = reinterpret_cast<float(*)[NT * kRows][kFeatures]>(smem);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[warp][8 * n + 2 * t + (i & 1)][g + 8 * (i >> 1)] = acc[n][i];
    __syncthreads();
    add_parts<NT>(a, f, n0, part);
}

// ---------------------------------------------------------------- 8 bits

__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A warp's step is one block of 128 k, whose sum gets its scales when it is
// complete: the weight's is one number for the 16 features, the rows' come two
// to a lane.  The codes go to the MMA as they lie, which unpacks them by instructions:
// 4.5 TB/s at most, so only the smallest calls come here.
__global__ void __launch_bounds__(kWarps * 32, 3) k_few_rows8(const FewArgs a)
{
    __shared__ float part[kWarps][kRows][kFeatures];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int li = blockIdx.x / a.blocks, n0 = (blockIdx.x - li * a.blocks) * kFeatures;
    dependents_may_launch();
    wait_for_prior_grid();
    int front, back;
    bool bad;
    const Found f = find_expert(a, li, front, back, bad);
    if (bad && blockIdx.x == 0 && threadIdx.x == 0) set_status(a.status, BSL_ERR_INVALID_ARG);
    if (a.zero_rest && li == 0) zero_rest_rows(a, n0, front, back);
    if (f.e < 0) return;

    const int64_t bytes = a.K;
    const bool in0 = n0 + g < a.N, in1 = n0 + g + 8 < a.N;
    const uint8_t *w0 = a.W + (static_cast<int64_t>(f.e) * a.N + n0 + g) * bytes + 16 * t, *w1 = w0 + 8 * bytes;
    const uint8_t *x = a.X + static_cast<int64_t>(f.first + g) * bytes + 16 * t;
    const int blocks = (a.K + 127) / 128;
    const float *ws = reinterpret_cast<const float *>(a.w_scales) +
                      (static_cast<int64_t>(f.e) * ((a.N + 127) / 128) + n0 / 128) * blocks;
    const float *xs = reinterpret_cast<const float *>(a.x_scales) + static_cast<int64_t>(f.first + 2 * t) * blocks;
    constexpr int U = 2;  // blocks on the way
    float acc[4] = {};
    for (int b0 = warp; b0 < blocks; b0 += kWarps * U) {
        uint4 va[U][2], vb[U][2], vx[U][2];
        float sw[U], sx[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int b = b0 + u * kWarps;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t at = static_cast<int64_t>(b) * 128 + 64 * h;
                const bool in = at + 16 * t < a.K;
                va[u][h] = vb[u][h] = make_uint4(0, 0, 0, 0);
                if (in && in0) va[u][h] = load_stream(w0 + at);
                if (in && in1) vb[u][h] = load_stream(w1 + at);
                vx[u][h] = make_uint4(0, 0, 0, 0);
                if (in && g < f.rows) vx[u][h] = load_global(reinterpret_cast<const uint4 *>(x + at));
            }
            sw[u] = b < blocks ? load_float(ws + b) : 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                sx[u][i] = b < blocks && 2 * t + i < f.rows ? load_float(xs + i * static_cast<int64_t>(blocks) + b) : 0.f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float c[4] = {};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                mma_e4m3(c, va[u][h].x, vb[u][h].x, va[u][h].y, vb[u][h].y, vx[u][h].x, vx[u][h].y);
                mma_e4m3(c, va[u][h].z, vb[u][h].z, va[u][h].w, vb[u][h].w, vx[u][h].z, vx[u][h].w);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] += c[i] * (sw[u] * sx[u][i & 1]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) part[warp][2 * t + (i & 1)][g + 8 * (i >> 1)] = acc[i];
    __syncthreads();
    add_parts<1>(a, f, n0, part);
}

bsl_status launch(void (*kern)(const FewArgs), FewArgs &a, int smem, cudaStream_t s)
{
    a.blocks = (a.N + kFeatures - 1) / kFeatures;
    const int64_t grid = static_cast<int64_t>(a.blocks) * (a.T < a.E ? a.T : a.E);
    if (grid > 0x7FFFFFFF) return BSL_ERR_UNSUPPORTED;
    return cuda_status(launch_dependent(kern, static_cast<unsigned>(grid), kWarps * 32, smem, s, a));
}

template <int NT>
bsl_status launch4(FewArgs &a, cudaStream_t s)
{
    static_assert(Few4<NT>::SMEM <= 48 * 1024, "no attribute needed");
    return launch(k_few_rows4<NT>, a, Few4<NT>::SMEM, s);
}

}  // namespace

// Where these kernels are ahead of the tensor-core tiles, by the rows and by the
// bytes of the weights that the rows can use (L2 cold; us here / there).
// Single calls behind other work also pay the tiles' set-up, some 5 us: there these stay ahead past each border
// (16 rows up to 64 MB, 32 rows up to 28 MB on one expert), or lose up to 7 % just below it (16 rows of 4 bits on
// eight experts, 4 MB: 14.3 / 13.3).
// bf16: up to 8 rows everywhere (17 MB 5.6 / 13.7, 361 MB 60 / 67, 721 MB 114 / 114); 16 rows re-read X for every
// 16 features, so up to 32 MB (17 MB 7.6 / 13.6, 34 MB 12.0 / 12.3, 90 MB 23.9 / 22.6); 32 rows up to 20 MB
// (17 MB 10.1 / 13.6, 34 MB 15.6 / 12.3).
bool few_rows(int32_t T, const bsl_grouped *W)
{
    const int64_t bytes = static_cast<int64_t>(T < W->E ? T : W->E) * W->N * W->K * 2;
    return T <= kRows || (T <= 2 * kRows && bytes <= (32ll << 20)) || (T <= 4 * kRows && bytes <= 20000000);
}

// 4 bits, products alone: 8 rows on 0.5 MB of codes 3.1 / 6.3, 8.4 MB 9.4 / 11.7, 22 MB 15.0 / 13.0; 16 rows on
// 0.5 MB 4.0 / 6.4, 4.2 MB 7.4 / 8.7, 8.4 MB 11.8 / 11.7.
bool few_rows4(int32_t T, const bsl_mx4 *W)
{
    const int64_t bytes = static_cast<int64_t>(T < W->E ? T : W->E) * W->N * (W->K / 2);
    return (T <= kRows && bytes <= (12ll << 20)) || (T <= 2 * kRows && bytes <= (4ll << 20));
}

// 8 bits, products alone, here / on the tensor-core tiles of few rows (fp8_few.cu): up to 8 rows on 1 MB 8.2 / 12.3,
// 17 MB 12.3 / 16.4, 45 MB 18.4 / 24.6, 361 MB on eight experts 80 / 84; 16 rows on 17 MB 18.4 / 16.4.
bool few_rows8(int32_t T) { return T <= kRows; }

bsl_status launch_few_rows(const void *X, int32_t T, const int32_t *offsets, const bsl_grouped *W, const void *bias,
                           void *Y, int32_t zero_rest, cudaStream_t s)
{
    FewArgs a = {static_cast<const uint8_t *>(W->weight), nullptr, static_cast<const uint8_t *>(X), nullptr,
                 static_cast<const __nv_bfloat16 *>(bias), static_cast<__nv_bfloat16 *>(Y), offsets, W->status,
                 T, W->E, W->N, W->K, 0, zero_rest};
    return launch(T <= kRows ? k_few_rows<1> : T <= 2 * kRows ? k_few_rows<2> : k_few_rows<4>, a, 0, s);
}

bsl_status launch_few_rows4(const uint8_t *xc, const uint8_t *xs, int32_t T, const int32_t *offsets, const bsl_mx4 *W,
                            const void *bias, void *Y, int32_t zero_rest, cudaStream_t s)
{
    FewArgs a = {W->codes, W->scales, xc, xs, static_cast<const __nv_bfloat16 *>(bias), static_cast<__nv_bfloat16 *>(Y),
                 offsets, W->status, T, W->E, W->N, W->K, 0, zero_rest};
    return T <= kRows ? launch4<1>(a, s) : launch4<2>(a, s);
}

bsl_status launch_few_rows8(const uint8_t *xc, const float *xs, int32_t T, const int32_t *offsets, const bsl_fp8 *W,
                            const void *bias, void *Y, int32_t zero_rest, cudaStream_t s)
{
    FewArgs a = {W->codes, reinterpret_cast<const uint8_t *>(W->scales), xc, reinterpret_cast<const uint8_t *>(xs),
                 static_cast<const __nv_bfloat16 *>(bias), static_cast<__nv_bfloat16 *>(Y), offsets, W->status,
                 T, W->E, W->N, W->K, 0, zero_rest};
    return launch(k_few_rows8, a, 0, s);
}

}  // namespace bsl
