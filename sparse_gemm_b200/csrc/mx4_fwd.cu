// mx4_fwd.cu -- product of two microscaled 4-bit matrices (mx4_quant.cu gives
// the format): Y = Q(X) . Q(W)^T + bias, dense or grouped by expert, fp32
// accumulation, one rounding to bf16.
#include "common.cuh"
#include "grouped.cuh"
#include "internal.h"

namespace bsl {
namespace {

constexpr int kTile = 32;

struct Mx4Args {
    const uint8_t *xc, *xs, *wc, *ws;
    const __nv_bfloat16 *bias;
    __nv_bfloat16 *Y;
    const int32_t *offsets;  // null: one group of all rows
    int32_t *status;
    int32_t T, E, N, K, zero_rest;
};

__device__ __forceinline__ float element(const uint8_t *codes, const uint8_t *scales, int64_t row, int k, int K)
{
    const uint32_t byte = codes[row * (K / 2) + k / 2], c = (k & 1) ? byte >> 4 : byte & 15u, m = c & 7u;
    const uint32_t b = scales[row * (K / 32) + k / 32];
    const float v = m < 2 ? 0.5f * static_cast<float>(m)
                          : __uint_as_float(((m >> 1) + 126u) << 23 | (m & 1u) << 22);
    return (c & 8u ? -v : v) * __uint_as_float(b == 255 ? 0x7FC00000u : b == 0 ? 0x00400000u : b << 23);
}

__global__ void k_mx4_plain(const Mx4Args a)
{
    __shared__ int32_t off[kMaxExperts + 1];
    __shared__ float sa[kTile][kTile + 1], sb[kTile][kTile + 1];
    if (a.offsets) {
        load_offsets(a.offsets, a.E, a.T, off, a.status);
    } else if (threadIdx.x == 0) {
        off[0] = 0;
        off[1] = a.T;
    }
    __syncthreads();
    const int tx = threadIdx.x % kTile, ty = threadIdx.x / kTile;
    const int c0 = blockIdx.y * kTile;
    int e, t = blockIdx.x;
    for (e = 0; e < a.E; ++e) {
        const int n = (off[e + 1] - off[e] + kTile - 1) / kTile;
        if (t < n) break;
        t -= n;
    }
    if (e == a.E) {
        if (!a.zero_rest) return;
        for (int64_t r = 0; t == 0 && r < a.T; ++r)
            if ((r < off[0] || r >= off[a.E]) && ty == 0 && c0 + tx < a.N)
                a.Y[r * a.N + c0 + tx] = __float2bfloat16(0.f);
        return;
    }
    const int r0 = off[e] + t * kTile, rend = off[e + 1];
    float acc = 0.f;
    for (int k0 = 0; k0 < a.K; k0 += kTile) {
        sa[ty][tx] = r0 + ty < rend ? element(a.xc, a.xs, r0 + ty, k0 + tx, a.K) : 0.f;
        sb[ty][tx] = c0 + ty < a.N ? element(a.wc, a.ws, static_cast<int64_t>(e) * a.N + c0 + ty, k0 + tx, a.K) : 0.f;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kTile; ++k) acc = fmaf(sa[ty][k], sb[tx][k], acc);
        __syncthreads();
    }
    if (r0 + ty < rend && c0 + tx < a.N) {
        if (a.bias) acc += __bfloat162float(a.bias[static_cast<int64_t>(e) * a.N + c0 + tx]);
        a.Y[static_cast<int64_t>(r0 + ty) * a.N + c0 + tx] = __float2bfloat16(acc);
    }
}

}  // namespace

bsl_status launch_mx4_fwd(const uint8_t *xc, const uint8_t *xs, int32_t T, const int32_t *offsets, const bsl_mx4 *W,
                          const void *bias, void *Y, int32_t zero_rest, cudaStream_t s)
{
    Mx4Args a = {xc, xs, W->codes, W->scales, static_cast<const __nv_bfloat16 *>(bias), static_cast<__nv_bfloat16 *>(Y),
                 offsets, W->status, T, W->E, W->N, W->K, zero_rest};
    const dim3 grid(T / kTile + W->E + 8, (W->N + kTile - 1) / kTile);
    k_mx4_plain<<<grid, kTile * kTile, 0, s>>>(a);
    return cuda_status(cudaGetLastError());
}

}  // namespace bsl
