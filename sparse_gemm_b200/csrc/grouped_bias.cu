// grouped_bias.cu -- bias gradient of the expert (grouped) linear layer:
//     db[e][n] = sum over the rows t of expert e of dY[t][n]
// in fp32, rounded once to bf16; an expert without rows gets zeros.
//
// As the dense layer's bias gradient (bias.cu): one CTA per 64-column tile and
// expert, 8 warps over the rows, partial sums added in warp order, so the
// result is identical run to run.  Bound by reading dY once.
#include "common.cuh"
#include "grouped.cuh"
#include "internal.h"

namespace bsl {
namespace {

constexpr int kWarps = 8;
constexpr int kCols = 64;  // columns per CTA: 2 per lane
constexpr int kLoads = 8;  // rows in flight per warp

__global__ void __launch_bounds__(kWarps * 32)
    k_grouped_bias_grad(const __nv_bfloat16 *__restrict__ dY, int32_t T, const int32_t *__restrict__ offsets, int32_t E,
                        int32_t N, __nv_bfloat16 *__restrict__ db)
{
    __shared__ int32_t off[kMaxExperts + 1];
    __shared__ float2 part[kWarps][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int e = blockIdx.y;
    const int col = blockIdx.x * kCols + 2 * lane;  // N is even: col and col + 1 are both inside or both outside
    load_offsets(offsets, E, T, off, nullptr);
    __syncthreads();
    float2 acc = make_float2(0.f, 0.f);
    if (col < N) {
        const __nv_bfloat162 *base = reinterpret_cast<const __nv_bfloat162 *>(dY + col);
        const int64_t stride = N / 2;
        const int end = off[e + 1];
        int m = off[e] + warp;
        for (; m + (kLoads - 1) * kWarps < end; m += kLoads * kWarps) {
            __nv_bfloat162 v[kLoads];
#pragma unroll
            for (int u = 0; u < kLoads; ++u) v[u] = base[static_cast<int64_t>(m + u * kWarps) * stride];
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                const float2 f = __bfloat1622float2(v[u]);
                acc.x += f.x;
                acc.y += f.y;
            }
        }
        for (; m < end; m += kWarps) {
            const float2 f = __bfloat1622float2(base[static_cast<int64_t>(m) * stride]);
            acc.x += f.x;
            acc.y += f.y;
        }
    }
    part[warp][lane] = acc;
    __syncthreads();
    if (warp == 0 && col < N) {
        float2 s = part[0][lane];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
            s.x += part[w][lane].x;
            s.y += part[w][lane].y;
        }
        reinterpret_cast<__nv_bfloat162 *>(db + static_cast<int64_t>(e) * N + col)[0] = __floats2bfloat162_rn(s.x, s.y);
    }
}

}  // namespace

bsl_status launch_grouped_bias_grad(const void *dY, int32_t T, const int32_t *offsets, int32_t E, int32_t N, void *db,
                                    cudaStream_t s)
{
    const dim3 grid((N + kCols - 1) / kCols, E);
    k_grouped_bias_grad<<<grid, kWarps * 32, 0, s>>>(static_cast<const __nv_bfloat16 *>(dY), T, offsets, E, N,
                                                      static_cast<__nv_bfloat16 *>(db));
    return cuda_status(cudaGetLastError());
}

}  // namespace bsl
