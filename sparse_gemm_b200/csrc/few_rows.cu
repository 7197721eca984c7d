// few_rows.cu -- forward of the expert (grouped) layer and of the 4-bit layer for
// a few rows in all (single tokens, up to 32): Y[t] = X[t] . W[e]^T + bias[e].
//
// Each weight row that is used is read once and little else matters: bytes and
// latency bound it.  A block owns 16 features of one expert and its 8 warps
// cut K, so that a call spreads over every SM at once, with no set-up before
// the first load but finding the block's expert.  A lane reads 16 bytes of a
// weight row at a time (two or four steps at once) and feeds them to mma.sync
// (m16n8k16, the rows of X on its N side) as they lie: the order of k inside
// a product is free as long as both operands share it.  The warps' fp32 sums
// are added in order through shared memory, and rounded once.
//
// 4-bit operands are turned into the bf16 numbers they stand for (mx4.cuh), five
// instructions for two codes.
#include "common.cuh"
#include "grouped.cuh"
#include "internal.h"
#include "mx4.cuh"

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

__device__ __forceinline__ uint4 load_stream(const void *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One step's products of 4-bit operands, NT groups of rows.
template <bool kHigh, int NT>
__device__ __forceinline__ void step4(float (&acc)[NT][4], const uint4 &a, const uint4 &b, const uint4 (&x)[NT],
                                      uint32_t sa, uint32_t sb, const uint32_t (&sx)[NT], uint32_t low)
{
    const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t p[4], q[4], r[4];
        decode8<kHigh>(aw[i], sa, low, p);
        decode8<kHigh>(bw[i], sb, low, q);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint32_t xw[4] = {x[n].x, x[n].y, x[n].z, x[n].w};
            decode8<kHigh>(xw[i], sx[n], low, r);
            mma_bf16(acc[n], p[0], q[0], p[1], q[1], r[0], r[1]);
            mma_bf16(acc[n], p[2], q[2], p[3], q[3], r[2], r[3]);
        }
    }
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
    const int raw0 = a.offsets[0];
    int carry = clamp(raw0), seen = 0;
    bad = carry != raw0;
    rest_front = carry;
    for (int i0 = 0; i0 < a.E; i0 += 32) {
        const int i = i0 + lane;
        const int raw = i < a.E ? a.offsets[i + 1] : 0;
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

// NT groups of eight rows: 1, 2 or 4 (bf16).
template <bool kF4, int NT>
__global__ void __launch_bounds__(kWarps * 32, kF4 && NT == 1 ? 4 : 3) k_few_rows(const FewArgs a)
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
    if (a.zero_rest && li == 0) {  // rows of no expert: the first expert's blocks, each its features
        const int n = n0 + threadIdx.x % kFeatures;
        for (int r = threadIdx.x / kFeatures; r < a.T; r += kWarps * 32 / kFeatures)
            if ((r < front || r >= back) && n < a.N) a.Y[static_cast<int64_t>(r) * a.N + n] = __float2bfloat16(0.f);
    }
    if (f.e < 0) return;

    // this lane's rows: features n0 + g and n0 + g + 8 of the weight, rows g, g + 8, ... of X
    constexpr int SPAN = kF4 ? 128 : 32;  // k of a step: 16 bytes a lane
    const int64_t bytes = kF4 ? a.K / 2 : static_cast<int64_t>(a.K) * 2;
    const int64_t wr = static_cast<int64_t>(f.e) * a.N + n0 + g;
    const bool in0 = n0 + g < a.N, in1 = n0 + g + 8 < a.N;
    const uint8_t *w0 = a.W + wr * bytes + 16 * t, *w1 = w0 + 8 * bytes;
    const uint8_t *x = a.X + static_cast<int64_t>(f.first + g) * bytes + 16 * t;
    const uint8_t *ws0 = kF4 ? a.w_scales + wr * (a.K / 32) + t : nullptr, *ws1 = kF4 ? ws0 + 8 * (a.K / 32) : nullptr;
    const uint8_t *xs = kF4 ? a.x_scales + static_cast<int64_t>(f.first + g) * (a.K / 32) + t : nullptr;
    const int steps = (a.K + SPAN - 1) / SPAN;
    constexpr int U = kF4 ? (NT == 1 ? 2 : 1) : NT == 4 ? 2 : 4;
    const int64_t scale_row = kF4 ? 8 * (a.K / 32) : 0;
    float acc[NT][4] = {};
    for (int s0 = warp; s0 < steps; s0 += kWarps * U) {
        uint4 va[U], vb[U], vx[U][NT];
        uint32_t sa[U], sb[U], sx[U][NT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = s0 + u * kWarps;
            const bool in = s * SPAN + t * (SPAN / 4) < a.K;
            va[u] = vb[u] = make_uint4(0, 0, 0, 0);
            sa[u] = sb[u] = 0;
            if (in && in0) va[u] = load_stream(w0 + static_cast<int64_t>(s) * 64);
            if (in && in1) vb[u] = load_stream(w1 + static_cast<int64_t>(s) * 64);
            if constexpr (kF4) {
                if (in && in0) sa[u] = __ldg(ws0 + 4 * s);
                if (in && in1) sb[u] = __ldg(ws1 + 4 * s);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                vx[u][n] = make_uint4(0, 0, 0, 0);
                sx[u][n] = 0;
                if (in && g + 8 * n < f.rows) {
                    vx[u][n] = __ldg(reinterpret_cast<const uint4 *>(x + n * 8 * bytes + static_cast<int64_t>(s) * 64));
                    if constexpr (kF4) sx[u][n] = __ldg(xs + n * scale_row + 4 * s);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if constexpr (kF4) {
                uint32_t top = max(sa[u], sb[u]);
#pragma unroll
                for (int n = 0; n < NT; ++n) top = max(top, sx[u][n]);
                // (255 stands for NaN whatever it is multiplied with)
                if (!__any_sync(0xffffffffu, top > 128)) {
                    step4<false, NT>(acc, va[u], vb[u], vx[u], sa[u], sb[u], sx[u], 0);
                } else {
                    // scales of 2^126 and 2^127: both operands 2^-4 of themselves, the products 2^8 of that
                    const bool far = __any_sync(0xffffffffu, top > 252);
                    float sum[NT][4] = {};
                    step4<true, NT>(sum, va[u], vb[u], vx[u], sa[u], sb[u], sx[u], far ? 4 : 0);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[n][i] += far ? 256.f * sum[n][i] : sum[n][i];
                }
            } else {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mma_bf16(acc[n], va[u].x, vb[u].x, va[u].y, vb[u].y, vx[u][n].x, vx[u][n].y);
                    mma_bf16(acc[n], va[u].z, vb[u].z, va[u].w, vb[u].w, vx[u][n].z, vx[u][n].w);
                }
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        part[warp][8 * n + 2 * t][g] = acc[n][0];
        part[warp][8 * n + 2 * t + 1][g] = acc[n][1];
        part[warp][8 * n + 2 * t][g + 8] = acc[n][2];
        part[warp][8 * n + 2 * t + 1][g + 8] = acc[n][3];
    }
    __syncthreads();
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

template <bool kF4>
bsl_status launch(FewArgs &a, cudaStream_t s)
{
    a.blocks = (a.N + kFeatures - 1) / kFeatures;
    const int64_t grid = static_cast<int64_t>(a.blocks) * (a.T < a.E ? a.T : a.E);
    if (grid > 0x7FFFFFFF) return BSL_ERR_UNSUPPORTED;
    const unsigned g = static_cast<unsigned>(grid);
    if (a.T <= kRows) return cuda_status(launch_dependent(k_few_rows<kF4, 1>, g, kWarps * 32, 0, s, a));
    if (kF4 || a.T <= 2 * kRows) return cuda_status(launch_dependent(k_few_rows<kF4, 2>, g, kWarps * 32, 0, s, a));
    return cuda_status(launch_dependent(k_few_rows<false, 4>, g, kWarps * 32, 0, s, a));
}

}  // namespace

// Where these kernels are ahead of the tensor-core tiles, by the rows and by the
// bytes of the weights that the rows can use (L2 cold; us here / there).
// bf16: up to 8 rows everywhere (17 MB 5.6 / 13.7, 361 MB 60 / 67, 721 MB 114 / 114); 16 rows re-read X for every
// 16 features, so up to 32 MB (17 MB 7.6 / 13.6, 34 MB 12.0 / 12.3, 90 MB 23.9 / 22.6); 32 rows up to 20 MB
// (17 MB 10.1 / 13.6, 34 MB 15.6 / 12.3).
bool few_rows(int32_t T, const bsl_grouped *W)
{
    const int64_t bytes = static_cast<int64_t>(T < W->E ? T : W->E) * W->N * W->K * 2;
    return T <= kRows || (T <= 2 * kRows && bytes <= (32ll << 20)) || (T <= 4 * kRows && bytes <= 20000000);
}

// 4 bits: turning codes into numbers bounds it (8 rows: 4.2 MB of codes 6.7 / 8.8, 8.4 MB 11.9 / 8.2, 22 MB
// 16.4 / 13.4; 16 rows: 0.3 MB 7.1 / 11.3, 4.2 MB 7.5 / 8.7, 8.4 MB 10.9 / 8.2).
bool few_rows4(int32_t T, const bsl_mx4 *W)
{
    const int64_t bytes = static_cast<int64_t>(T < W->E ? T : W->E) * W->N * (W->K / 2);
    return T <= 2 * kRows && bytes <= (4ll << 20);
}

bsl_status launch_few_rows(const void *X, int32_t T, const int32_t *offsets, const bsl_grouped *W, const void *bias,
                           void *Y, int32_t zero_rest, cudaStream_t s)
{
    FewArgs a = {static_cast<const uint8_t *>(W->weight), nullptr, static_cast<const uint8_t *>(X), nullptr,
                 static_cast<const __nv_bfloat16 *>(bias), static_cast<__nv_bfloat16 *>(Y), offsets, W->status,
                 T, W->E, W->N, W->K, 0, zero_rest};
    return launch<false>(a, s);
}

bsl_status launch_few_rows4(const uint8_t *xc, const uint8_t *xs, int32_t T, const int32_t *offsets, const bsl_mx4 *W,
                            const void *bias, void *Y, int32_t zero_rest, cudaStream_t s)
{
    FewArgs a = {W->codes, W->scales, xc, xs, static_cast<const __nv_bfloat16 *>(bias), static_cast<__nv_bfloat16 *>(Y),
                 offsets, W->status, T, W->E, W->N, W->K, 0, zero_rest};
    return launch<true>(a, s);
}

}  // namespace bsl
