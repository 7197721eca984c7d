// grouped.cu -- expert (grouped) linear layer: forward, input gradient and weight
// gradient on the kernel of grouped_kernel.cuh, and the weight gradient's
// per-expert tensor maps.
#include "grouped_kernel.cuh"

namespace bsl {
namespace {

// ------------------------------------------------------------ per-expert maps

// maps[e] = tensor maps of dY, X (one strip a copy), dY, X (two strips) that
// begin at the expert's first row and end with its last (an expert without
// rows keeps one row, never read).  One warp per expert: the template's copy
// in shared memory gets the address and the row count, then goes to global
// memory with the fence that TMA needs.
struct ExpertMaps {
    CUtensorMap m[4];
};

__global__ void __launch_bounds__(32)
    k_expert_maps(const __grid_constant__ ExpertMaps base, const void *dY, const void *X, int32_t N, int32_t K,
                  const int32_t *offsets, int32_t E, int32_t T, CUtensorMap *maps, int32_t *status)
{
    __shared__ int32_t off[kMaxExperts + 1];
    __shared__ alignas(128) CUtensorMap m[4];
    dependents_may_launch();
    wait_for_prior_grid();
    fetch_offsets(offsets, E, T, off);
    __syncwarp();
    clamp_offsets(E, T, off, blockIdx.x == 0 ? status : nullptr);
    const int lane = threadIdx.x, e = blockIdx.x;
    const int rows = off[e + 1] - off[e];
    uint32_t *w = reinterpret_cast<uint32_t *>(m);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[32 * i + lane] = reinterpret_cast<const uint32_t *>(&base.m[i])[lane];
    __syncwarp();
    if (lane < 4) {
        const uint32_t a = smem_u32(&m[lane]);
        const int64_t first = rows ? off[e] : 0;
        const char *p = lane & 1 ? static_cast<const char *>(X) + first * K * 2 : static_cast<const char *>(dY) + first * N * 2;
        asm volatile("tensormap.replace.tile.global_address.shared::cta.b1024.b64 [%0], %1;" ::"r"(a),
                     "l"(__cvta_generic_to_global(p))
                     : "memory");
        asm volatile("tensormap.replace.tile.global_dim.shared::cta.b1024.b32 [%0], 1, %1;" ::"r"(a), "r"(rows ? rows : 1)
                     : "memory");
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm volatile(
            "tensormap.cp_fenceproxy.global.shared::cta.tensormap::generic.release.gpu.sync.aligned [%0], [%1], 128;" ::"l"(
                __cvta_generic_to_global(maps + 4 * static_cast<size_t>(e) + i)),
            "r"(smem_u32(&m[i]))
            : "memory");
}

}  // namespace

size_t grouped_workspace_bytes(const bsl_grouped *W) { return static_cast<size_t>(W->E) * 4 * sizeof(CUtensorMap); }

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
                             void *dW, void *workspace, cudaStream_t s)
{
    const int64_t N = W->N, K = W->K;
    Maps m;
    ExpertMaps base;
    if (!map_rows(&base.m[0], dY, N, T, 64, 128, 128) || !map_rows(&base.m[1], X, K, T, 64, 128, 128) ||
        !make_strip_map(&base.m[2], dY, N, T, 1, 128, 2) || !make_strip_map(&base.m[3], X, K, T, 1, 128, 2) ||
        !make_map_3d(&m.out, dW, K, N, W->E, K * 2, K * 2 * N, 32, 32, 0))
        return BSL_ERR_CUDA;
    m.a[0] = base.m[2];  // (prefetched by every kernel)
    CUtensorMap *maps = static_cast<CUtensorMap *>(workspace);
    const bsl_status st = cuda_status(launch_dependent(k_expert_maps, W->E, 32, 0, s, base, dY, X, W->N, W->K, offsets,
                                                       W->E, T, maps, W->status));
    if (st != BSL_OK) return st;
    Args args = {};
    args.offsets = offsets;
    args.expert_maps = maps;
    args.T = T;
    args.E = W->E;
    args.cols = W->K;
    args.rows = W->N;
    args.status = W->status;
    args.timeout_ns = wait_timeout_ns();
    return run<kWeightGrad>(m, args, s);
}

}  // namespace bsl
