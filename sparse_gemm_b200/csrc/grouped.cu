// grouped.cu -- expert (grouped) linear layer: one weight per group of rows.
//
// The rows of X are sorted by expert: rows offsets[e] .. offsets[e+1] - 1 are
// multiplied with expert e's weight W[e] [N][K]:
//     forward          Y[t]  = X[t] . W[e]^T + bias[e]
//     input gradient   dX[t] = dY[t] . W[e]
//     weight gradient  dW[e] = sum over the rows t of e of dY[t]^T . X[t]
//     bias gradient    db[e] = sum over the rows t of e of dY[t]
// (bf16 in, fp32 accumulation, one rounding to bf16).
#include "common.cuh"
#include "grouped.cuh"
#include "internal.h"

namespace bsl {
namespace {

constexpr int kTile = 32;  // rows and columns of an output tile

struct GroupedArgs {
    const __nv_bfloat16 *A, *B, *bias;
    __nv_bfloat16 *out;
    const int32_t *offsets;
    int32_t *status;
    int32_t T, E;
    int32_t rows, cols, depth;  // of one expert's product; the ragged one is unused
    int32_t zero_rest;
};

// out[r][c] = sum_k A(r, k) B(c, k).  kMode 0: forward, 1: input gradient,
// 2: weight gradient (r = output feature, k = row of the group).
template <int kMode>
__global__ void k_grouped_plain(const GroupedArgs a)
{
    __shared__ int32_t off[kMaxExperts + 1];
    __shared__ float sa[kTile][kTile + 1], sb[kTile][kTile + 1];
    load_offsets(a.offsets, a.E, a.T, off, a.status);
    __syncthreads();
    const int tx = threadIdx.x % kTile, ty = threadIdx.x / kTile;
    const int c0 = blockIdx.y * kTile;
    int e, r0, rend;
    if (kMode == 2) {
        e = blockIdx.z;
        r0 = blockIdx.x * kTile;
        rend = a.rows;
    } else {
        int t = blockIdx.x;
        for (e = 0; e < a.E; ++e) {
            const int n = (off[e + 1] - off[e] + kTile - 1) / kTile;
            if (t < n) break;
            t -= n;
        }
        if (e == a.E) {  // rows of no expert
            if (!a.zero_rest) return;
            for (int64_t r = 0; t == 0 && r < a.T; ++r)
                if ((r < off[0] || r >= off[a.E]) && ty == 0 && c0 + tx < a.cols)
                    a.out[r * a.cols + c0 + tx] = __float2bfloat16(0.f);
            return;
        }
        r0 = off[e] + t * kTile;
        rend = off[e + 1];
    }
    const int depth = kMode == 2 ? off[e + 1] - off[e] : a.depth;
    float acc = 0.f;
    for (int k0 = 0; k0 < depth; k0 += kTile) {
        float va = 0.f, vb = 0.f;
        if (kMode == 2) {  // ty: k, tx: row or column
            const int64_t t = off[e] + k0 + ty;
            if (k0 + ty < depth && r0 + tx < rend) va = __bfloat162float(a.A[t * a.rows + r0 + tx]);
            if (k0 + ty < depth && c0 + tx < a.cols) vb = __bfloat162float(a.B[t * a.cols + c0 + tx]);
            sa[tx][ty] = va;
            sb[tx][ty] = vb;
        } else {
            if (r0 + ty < rend && k0 + tx < depth) va = __bfloat162float(a.A[static_cast<int64_t>(r0 + ty) * depth + k0 + tx]);
            sa[ty][tx] = va;
            const __nv_bfloat16 *w = a.B + static_cast<int64_t>(e) * a.cols * depth;
            if (kMode == 0) {
                if (c0 + ty < a.cols && k0 + tx < depth) vb = __bfloat162float(w[static_cast<int64_t>(c0 + ty) * depth + k0 + tx]);
                sb[ty][tx] = vb;
            } else {
                if (k0 + ty < depth && c0 + tx < a.cols) vb = __bfloat162float(w[static_cast<int64_t>(k0 + ty) * a.cols + c0 + tx]);
                sb[tx][ty] = vb;
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kTile; ++k) acc = fmaf(sa[ty][k], sb[tx][k], acc);
        __syncthreads();
    }
    if (r0 + ty < rend && c0 + tx < a.cols) {
        if (a.bias) acc += __bfloat162float(a.bias[static_cast<int64_t>(e) * a.cols + c0 + tx]);
        const int64_t row = kMode == 2 ? static_cast<int64_t>(e) * a.rows + r0 + ty : r0 + ty;
        a.out[row * a.cols + c0 + tx] = __float2bfloat16(acc);
    }
}

}  // namespace

size_t grouped_workspace_bytes(const bsl_grouped *) { return 0; }

bsl_status launch_grouped_rows(const void *A, int32_t T, const int32_t *offsets, const bsl_grouped *W, bool transposed,
                               const void *bias, void *out, int32_t zero_rest, cudaStream_t s)
{
    GroupedArgs a = {};
    a.A = static_cast<const __nv_bfloat16 *>(A);
    a.B = static_cast<const __nv_bfloat16 *>(W->weight);
    a.bias = static_cast<const __nv_bfloat16 *>(bias);
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.offsets = offsets;
    a.status = W->status;
    a.T = T;
    a.E = W->E;
    a.cols = transposed ? W->K : W->N;
    a.depth = transposed ? W->N : W->K;
    a.zero_rest = zero_rest;
    const dim3 grid(T / kTile + W->E + 8, (a.cols + kTile - 1) / kTile);
    if (transposed) k_grouped_plain<1><<<grid, kTile * kTile, 0, s>>>(a);
    else k_grouped_plain<0><<<grid, kTile * kTile, 0, s>>>(a);
    return cuda_status(cudaGetLastError());
}

bsl_status launch_grouped_dw(const void *dY, const void *X, int32_t T, const int32_t *offsets, const bsl_grouped *W,
                             void *dW, void *, cudaStream_t s)
{
    GroupedArgs a = {};
    a.A = static_cast<const __nv_bfloat16 *>(dY);
    a.B = static_cast<const __nv_bfloat16 *>(X);
    a.out = static_cast<__nv_bfloat16 *>(dW);
    a.offsets = offsets;
    a.status = W->status;
    a.T = T;
    a.E = W->E;
    a.rows = W->N;
    a.cols = W->K;
    const dim3 grid((W->N + kTile - 1) / kTile, (W->K + kTile - 1) / kTile, W->E);
    k_grouped_plain<2><<<grid, kTile * kTile, 0, s>>>(a);
    return cuda_status(cudaGetLastError());
}

}  // namespace bsl
