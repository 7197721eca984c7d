// mx4_fwd.cu -- product of two microscaled 4-bit matrices (mx4_quant.cu gives
// the format): Y = Q(X) . Q(W)^T + bias, dense or grouped by expert, on the
// block-scaled MMA of grouped_kernel.cuh.
//
// To the copies a row of K 4-bit codes is a row of K / 4 two-byte columns, so
// the tiles, boxes and tails are those of the bf16 forward with a depth of
// K / 4; 32 bytes of a row are 64 elements, one K step of the MMA.
#include "grouped_kernel.cuh"

namespace bsl {

bsl_status launch_mx4_fwd(const uint8_t *xc, const uint8_t *xs, int32_t T, const int32_t *offsets, const bsl_mx4 *W,
                          const void *bias, void *Y, int32_t zero_rest, cudaStream_t s)
{
    if (few_rows4(T, W)) return launch_few_rows4(xc, xs, T, offsets, W, bias, Y, zero_rest, s);
    Args args = {};
    args.offsets = offsets;
    args.bias = static_cast<const __nv_bfloat16 *>(bias);
    args.out = static_cast<__nv_bfloat16 *>(Y);
    args.status = W->status;
    args.T = T;
    args.E = W->E;
    args.cols = W->N;
    args.depth = W->K / 4;
    args.zero_rest = zero_rest;
    args.a_scales = W->scales;
    args.b_scales = xs;
    args.scale_bytes = W->K / 32;
    args.timeout_ns = wait_timeout_ns();
    Maps m;
    if (!row_maps(m, W->codes, W->E, W->N, args.depth, xc, T, args.depth, Y, W->N)) return BSL_ERR_CUDA;
    if (W->K % 512 == 0) return run<kForward4>(m, args, s);
    if (W->K % 256 == 0) return run<kForward4By8>(m, args, s);
    return W->K % 128 == 0 ? run<kForward4By4>(m, args, s) : run<kForward4Any>(m, args, s);
}

}  // namespace bsl
