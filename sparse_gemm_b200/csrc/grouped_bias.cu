// grouped_bias.cu -- bias gradient of the expert (grouped) linear layer:
//     db[e][n] = sum over the rows t of expert e of dY[t][n]
// in fp32, rounded once to bf16; an expert without rows gets zeros.
//
// Bound by reading dY once.  A cluster of S CTAs owns 256 columns of one
// expert (16 bytes a lane, 512 bytes of a row a warp) and cuts the expert's
// rows into S equal parts; inside a CTA the 8 warps take rows w, w + 8, ...
// with 8 loads in flight.  Warps are added in order through shared memory,
// CTAs in order through distributed shared memory, so the result is identical
// run to run and needs no scratch.
//
// S (1 .. 8) brings a CTA down to 512 rows, further, to 128 at least, while
// there are fewer CTAs than the GPU holds at a time.  16384 rows x 14336
// columns: 77 us (6.1 TB/s) for one expert and for eight; unsplit 1140 and 306.
// 8192 rows of eight experts: 44 us with 256 rows a CTA, 54 with 128, 47 with 512.
#include "common.cuh"
#include "grouped.cuh"
#include "internal.h"

namespace bsl {
namespace {

constexpr int kWarps = 8;
constexpr int kCols = 256;  // columns per CTA: 8 per lane
constexpr int kLoads = 8;   // rows in flight per warp

__device__ __forceinline__ void add8(float (&acc)[8], const uint4 &v)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        acc[2 * i] += __uint_as_float(w[i] << 16);
        acc[2 * i + 1] += __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__global__ void __launch_bounds__(kWarps * 32)
    k_grouped_bias_grad(const uint4 *dY, int32_t T, const int32_t *offsets, int32_t E, int32_t N, int32_t S,
                        __nv_bfloat16 *db)
{
    __shared__ int32_t off[kMaxExperts + 1];
    __shared__ float part[kWarps][kCols];
    __shared__ float sum[kCols];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = blockIdx.x % S, cols = blockIdx.x / S;
    const int tiles = (N + kCols - 1) / kCols;
    const int e = cols / tiles;
    const int col = (cols - e * tiles) * kCols + 8 * lane;  // N is a multiple of 8
    dependents_may_launch();
    wait_for_prior_grid();
    fetch_offsets(offsets, E, T, off);
    __syncthreads();
    if (warp == 0) clamp_offsets(E, T, off, nullptr);
    __syncthreads();
    float acc[8] = {};
    if (col < N) {
        const int64_t rows = off[e + 1] - off[e];
        const int end = off[e] + static_cast<int>(rows * (rank + 1) / S);
        int m = off[e] + static_cast<int>(rows * rank / S) + warp;
        const uint4 *base = dY + col / 8;
        const int64_t stride = N / 8;
        for (; m + (kLoads - 1) * kWarps < end; m += kLoads * kWarps) {
            uint4 v[kLoads];
#pragma unroll
            for (int u = 0; u < kLoads; ++u) v[u] = load_global(base + static_cast<int64_t>(m + u * kWarps) * stride);
#pragma unroll
            for (int u = 0; u < kLoads; ++u) add8(acc, v[u]);
        }
        for (; m < end; m += kWarps) add8(acc, load_global(base + static_cast<int64_t>(m) * stride));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) part[warp][i * 32 + lane] = acc[i];  // column 8 * lane + i
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += part[w][threadIdx.x];
    sum[threadIdx.x] = s;
    cluster_sync_all();
    // rank r finishes every S-th group of columns
    const int c = (cols - e * tiles) * kCols + 8 * (threadIdx.x & 31) + (threadIdx.x >> 5);
    if ((threadIdx.x >> 5) % S == rank && c < N) {
        float t = 0.f;
        for (int r = 0; r < S; ++r) {
            float v;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr(&sum[threadIdx.x], r)));
            t += v;
        }
        db[static_cast<int64_t>(e) * N + c] = __float2bfloat16(t);
    }
    cluster_sync_all();  // no CTA ends while its sums are read
}

}  // namespace

bsl_status launch_grouped_bias_grad(const void *dY, int32_t T, const int32_t *offsets, int32_t E, int32_t N, void *db,
                                    cudaStream_t s)
{
    const int64_t tiles = static_cast<int64_t>((N + kCols - 1) / kCols) * E;
    int32_t S = 1;
    while (S < 8 && (static_cast<int64_t>(E) * S * 512 < T ||
                     (tiles * S < 7 * num_sms() && static_cast<int64_t>(E) * S * 128 < T)))
        S *= 2;
    const int64_t grid = tiles * S;
    if (grid > 0x7FFFFFFF) return BSL_ERR_UNSUPPORTED;
    return cuda_status(launch_dependent_cluster(k_grouped_bias_grad, static_cast<unsigned>(grid), S, kWarps * 32, 0, s,
                                                static_cast<const uint4 *>(dY), T, offsets, E, N, S,
                                                static_cast<__nv_bfloat16 *>(db)));
}

}  // namespace bsl
