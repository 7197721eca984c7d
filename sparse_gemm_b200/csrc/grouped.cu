// grouped.cu -- expert (grouped) linear layer: forward, input gradient and weight
// gradient on the kernel of grouped_kernel.cuh.
#include "grouped_kernel.cuh"

namespace bsl {

bsl_status launch_grouped_rows(const void *A, int32_t T, const int32_t *offsets, const bsl_grouped *W, bool transposed,
                               const void *bias, void *out, int32_t zero_rest, cudaStream_t s)
{
    if (!transposed && few_rows(T, W)) return launch_few_rows(A, T, offsets, W, bias, out, zero_rest, s);
    Args args = {};
    args.offsets = offsets;
    args.bias = static_cast<const __nv_bfloat16 *>(bias);
    args.out = static_cast<__nv_bfloat16 *>(out);
    args.status = W->status;
    args.T = T;
    args.E = W->E;
    args.cols = transposed ? W->K : W->N;
    args.depth = transposed ? W->N : W->K;
    args.zero_rest = zero_rest;
    args.timeout_ns = wait_timeout_ns();
    Maps m;
    if (!row_maps(m, W->weight, W->E, W->N, W->K, A, T, args.depth, out, args.cols)) return BSL_ERR_CUDA;
    return transposed ? run<kInputGrad>(m, args, s) : run<kForward>(m, args, s);
}

bsl_status launch_grouped_dw(const void *dY, const void *X, int32_t T, const int32_t *offsets, const bsl_grouped *W,
                             void *dW, cudaStream_t s)
{
    const int64_t N = W->N, K = W->K;
    Maps m;
    bool good = make_strip_map(&m.a[0], X, K, T, 1, 128, 2) && map_rows(&m.a[1], X, K, T, 64, 128, 128) &&
                make_strip_map(&m.b[0], dY, N, T, 1, 128, 2) && map_rows(&m.b[1], dY, N, T, 64, 128, 128) &&
                make_map_3d(&m.out, dW, K, N, W->E, K * 2, K * 2 * N, 32, 32, 0);
    for (int j = 0; j < 7; ++j)
        good = good && map_rows(&m.b[2 + j], dY, N, T, 64, 64 >> j, 128) && map_rows(&m.b[9 + j], X, K, T, 64, 64 >> j, 128);
    if (!good) return BSL_ERR_CUDA;
    Args args = {};
    args.offsets = offsets;
    args.T = T;
    args.E = W->E;
    args.cols = W->K;
    args.rows = W->N;
    args.status = W->status;
    args.timeout_ns = wait_timeout_ns();
    return run<kWeightGrad>(m, args, s);
}

}  // namespace bsl
