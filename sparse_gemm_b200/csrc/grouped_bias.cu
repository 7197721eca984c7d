// grouped_bias.cu -- bias gradient of the expert (grouped) linear layer:
//     db[e][n] = sum over the rows t of expert e of dY[t][n]
// in fp32, rounded once to bf16; an expert without rows gets zeros.
//
// Bound by reading dY once.  A cluster owns 256 columns (16 bytes a lane, 512
// bytes of a row a warp).  Where experts are few it has one of them and S CTAs,
// which cut the expert's rows into equal parts.  Where they are many (S = 1)
// it has G experts and as many CTAs, one for each expert; but one with more
// than `most` rows is cut over all G first: the offsets are known on the device
// only, and one expert may hold nearly all rows.  Inside a CTA the 8 warps
// take rows w, w + 8, ... with 8 loads in flight.  Warps are added in order
// through shared memory, CTAs in order through distributed shared memory, so
// the result is identical run to run and needs no scratch.
//
// S (1 .. 8) brings a CTA down to 512 rows if the shares are equal, further,
// to 128 at least, while there are fewer CTAs than the GPU holds at a time.
// Measured, calls in a row: 16384 rows x 14336 columns 69 us for one expert, 80 for
// eight, 83 for 64; with 90 % of the rows in one expert 86 us of eight (S = 4), 145
// of 16 (S = 2), 82 of 64 (412 with one CTA for it).  8192 rows of eight
// experts: 46 us with 256 rows a CTA; with 128 and 512 it lost 10 and 3 us.  G
// experts with S = 2 or 4 CTAs each, which then all wait for the cluster's
// slowest: 90 % in one of 16 would take 110 instead of 152 us (L2 cold), but
// mildly uneven shares 112 instead of 104.  64 registers a thread (four CTAs an
// SM) keep the 8 loads in flight; with 42, as the compiler would have it, one
// expert takes 88 instead of 45 us at 16384 x 4096.
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

// This CTA's part (`part` of `parts`) of the sums over an expert's rows, into sum[256].
__device__ __forceinline__ void sum_rows(const uint4 *dY, int32_t N, int first, int64_t rows, int part, int parts, int col,
                                         float (*warps)[kCols], float *sum)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float acc[8] = {};
    if (col < N) {
        const int end = first + static_cast<int>(rows * (part + 1) / parts);
        int m = first + static_cast<int>(rows * part / parts) + warp;
        const uint4 *base = dY + col / 8;
        const int64_t stride = N / 8;
        for (; m + (kLoads - 1) * kWarps < end; m += kLoads * kWarps) {
            uint4 v[kLoads];
#pragma unroll
            for (int u = 0; u < kLoads; ++u) v[u] = load_stream(base + static_cast<int64_t>(m + u * kWarps) * stride);
#pragma unroll
            for (int u = 0; u < kLoads; ++u) add8(acc, v[u]);
        }
        for (; m < end; m += kWarps) add8(acc, load_stream(base + static_cast<int64_t>(m) * stride));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) warps[warp][i * 32 + lane] = acc[i];  // column 8 * lane + i
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += warps[w][threadIdx.x];
    sum[threadIdx.x] = s;
}

__global__ void __launch_bounds__(kWarps * 32, 4)
    k_grouped_bias_grad(const uint4 *dY, int32_t T, const int32_t *offsets, int32_t E, int32_t N, int32_t C, int32_t G,
                        int32_t most, __nv_bfloat16 *db)
{
    __shared__ int32_t off[kMaxExperts + 1];
    __shared__ float warps[kWarps][kCols];
    __shared__ float sum[kCols];
    const int rank = blockIdx.x % C, unit = blockIdx.x / C;
    const int tiles = (N + kCols - 1) / kCols;
    const int group = unit / tiles;
    const int col0 = (unit - group * tiles) * kCols, col = col0 + 8 * (threadIdx.x & 31);  // N is a multiple of 8
    dependents_may_launch();
    wait_for_prior_grid();
    fetch_offsets(offsets, E, T, off);
    __syncthreads();
    if (threadIdx.x < 32) clamp_offsets(E, T, off, nullptr);
    __syncthreads();
    const int e0 = group * G, e1 = e0 + G < E ? e0 + G : E;
    auto rows_of = [&](int e) { return off[e + 1] - off[e]; };
    for (int next = e0;; ++next) {
        // first the experts that the cluster shares, the same in all its CTAs, which so meet at every barrier
        while (G > 1 && next < e1 && rows_of(next) <= most) ++next;
        const bool shared = next < e1;
        const int e = shared ? next : e0 + rank;
        if (!shared && (G == 1 || e >= e1 || rows_of(e) > most)) break;
        const int parts = shared ? C : 1, part = shared ? rank : 0;
        sum_rows(dY, N, off[e], rows_of(e), part, parts, col, warps, sum);
        if (shared) cluster_sync_all();
        // rank r finishes every parts-th group of columns
        const int c = col0 + 8 * (threadIdx.x & 31) + (threadIdx.x >> 5);
        if ((threadIdx.x >> 5) % parts == part && c < N) {
            float t = 0.f;
            for (int r = 0; r < parts; ++r) {
                float v;
                asm volatile("ld.shared::cluster.f32 %0, [%1];"
                             : "=f"(v)
                             : "r"(cluster_addr(&sum[threadIdx.x], shared ? r : rank)));
                t += v;
            }
            db[static_cast<int64_t>(e) * N + c] = __float2bfloat16(t);
        }
        if (!shared) break;  // then a CTA for each of the others, which waits for no one
        cluster_sync_all();  // the sums were read
    }
}

}  // namespace

bsl_status launch_grouped_bias_grad(const void *dY, int32_t T, const int32_t *offsets, int32_t E, int32_t N, void *db,
                                    cudaStream_t s)
{
    const int64_t tiles = (N + kCols - 1) / kCols;
    int32_t S = 1;
    while (S < 8 && (static_cast<int64_t>(E) * S * 512 < T ||
                     (tiles * E * S < 7 * num_sms() && static_cast<int64_t>(E) * S * 128 < T)))
        S *= 2;
    // (more than one CTA an expert would all wait for the cluster's slowest: mild skew costs more than it gives)
    int32_t G = 1;
    while (S == 1 && G < 8 && G < E && G * 512 < T) G *= 2;
    const int32_t C = S * G, groups = (E + G - 1) / G;
    // twice an equal share, and 512 rows at least (not looked at where G is 1)
    const int32_t share = T / E, most = G == 1 ? 0 : 2 * (share > 256 ? share : 256);
    const int64_t grid = tiles * groups * C;
    if (grid > 0x7FFFFFFF) return BSL_ERR_UNSUPPORTED;
    return cuda_status(launch_dependent_cluster(k_grouped_bias_grad, static_cast<unsigned>(grid), C, kWarps * 32, 0, s,
                                                static_cast<const uint4 *>(dY), T, offsets, E, N, C, G, most,
                                                static_cast<__nv_bfloat16 *>(db)));
}

}  // namespace bsl
