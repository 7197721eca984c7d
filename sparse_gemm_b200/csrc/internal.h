// internal.h -- host-side declarations shared by the libbsl translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <utility>

#include "bsl.h"

namespace bsl {

// Encode a 2-D bf16 tensor map: `inner` contiguous elements per row, `outer`
// rows, `row_bytes` between rows, box of box_inner x box_outer elements.
// swizzle_bytes: 0, 64 or 128.  Returns false if the driver rejects it.
bool make_map_2d(CUtensorMap *map, const void *base, uint64_t inner, uint64_t outer, uint64_t row_bytes,
                 uint32_t box_inner, uint32_t box_outer, int swizzle_bytes);

// Encode a 3-D bf16 tensor map: d0 contiguous elements, d1 rows `stride1`
// bytes apart, d2 planes `stride2` bytes apart; box of box0 x box1 x 1.
bool make_map_3d(CUtensorMap *map, const void *base, uint64_t d0, uint64_t d1, uint64_t d2, uint64_t stride1,
                 uint64_t stride2, uint32_t box0, uint32_t box1, int swizzle_bytes);

// Encode the strips of bf16 planes [planes][rows][cols] as a 4-D tensor map (x = column inside a strip of 64,
// y = row, z = strip, w = plane) with a box of 64 columns x box_rows rows x box_strips strips, 128-byte swizzle:
// one copy brings box_rows rows of 64 * box_strips columns, strip after strip of 128-byte rows.  Whole strips
// only (cols / 64 of them).  Strides need not grow from dimension to dimension: what lies outside is told
// coordinate by coordinate, and is neither read (fewer L2 sectors by as much) nor part of the result.
bool make_strip_map(CUtensorMap *map, const void *base, uint64_t cols, uint64_t rows, uint64_t planes,
                    uint32_t box_rows, uint32_t box_strips);

// Encode the packed weight values bf16 [nblocks][b][b] as a 3-D tensor map
// (x = column inside a block, y = row inside a block, z = block) with a
// box of b columns x box_rows rows x 1 block, swizzled like the kernels'
// shared-memory operands (128-byte rows for b = 64, 64-byte rows for b = 32).
bool make_block_map(CUtensorMap *map, const void *values, int32_t b, int32_t nblocks, uint32_t box_rows);

int num_sms();
// Argument and device checks shared by the entry points (api.cu).
bsl_status bind_device(const void *p);  // make the device owning p current

// Makes the device owning a pointer current for the duration of an entry
// point and puts the caller's current device back when it goes out of scope.
class DeviceGuard {
public:
    DeviceGuard() { cudaGetDevice(&prev_); }
    ~DeviceGuard()
    {
        int now = -1;
        if (cudaGetDevice(&now) == cudaSuccess && now != prev_) cudaSetDevice(prev_);
    }
    bsl_status bind(const void *p) { return bind_device(p); }
    DeviceGuard(const DeviceGuard &) = delete;
    DeviceGuard &operator=(const DeviceGuard &) = delete;

private:
    int prev_ = 0;
};

// Launch a kernel that may begin while the previous kernel in the stream is
// finishing (programmatic stream serialization).  The kernel must wait for
// the prior grid (wait_for_prior_grid, common.cuh) before its first global
// memory access; results and ordering are those of a plain launch.
template <typename... KArgs, typename... Args>
cudaError_t launch_dependent(void (*kern)(KArgs...), unsigned grid, unsigned block, size_t smem, cudaStream_t s,
                             Args &&...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

// The same with the grid cut into clusters of `cluster` CTAs (grid is a multiple of it).
template <typename... KArgs, typename... Args>
cudaError_t launch_dependent_cluster(void (*kern)(KArgs...), unsigned grid, unsigned cluster, unsigned block,
                                     size_t smem, cudaStream_t s, Args &&...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

// cudaFuncSetAttribute(MaxDynamicSharedMemorySize) once per kernel and device.
bsl_status set_smem_once(const void *func, int bytes);
bsl_status check_device();              // current device is sm_100
bsl_status check_bsr(const bsl_bsr *W);
bsl_status check_semi24(const bsl_semi24 *W);
bsl_status check_grouped(const bsl_grouped *W);
bsl_status check_mx4(const bsl_mx4 *W);
bsl_status check_fp8(const bsl_fp8 *W);
uint64_t wait_timeout_ns();
bsl_status cuda_status(cudaError_t e);
void note_driver_error(int code);

// Kernel launchers (defined next to their kernels).
bsl_status launch_pack(const void *W, const uint8_t *mask, const bsl_bsr *out, cudaStream_t s);
bsl_status launch_pack_count(const uint8_t *mask, int32_t R, int32_t C, int32_t *row_ptr, cudaStream_t s);

// Forward (A = X, segments = block rows) and input gradient (A = dY,
// segments = block columns through the CSC index) share one engine.
// bias: bf16 [out_cols] added to every output row (forward only; may be null).
bsl_status launch_spmm_tc(const void *A, int32_t M, int32_t a_cols, const bsl_bsr *W, bool transposed,
                          const void *bias, void *out, int32_t out_cols, cudaStream_t s);

bsl_status launch_sddmm_tc(const void *dY, const void *X, int32_t M, const bsl_bsr *W, void *dW,
                           cudaStream_t s);

size_t stream_workspace_bytes(int32_t M, const bsl_bsr *W);
bsl_status launch_stream_fwd(const void *X, int32_t M, const bsl_bsr *W, const void *bias, void *Y, void *ws,
                             cudaStream_t s);
bsl_status launch_bias_grad(const void *dY, int32_t M, int32_t N, void *dbias, cudaStream_t s);

// 2:4 semi-structured weight: compress a dense weight, forward on the sparse MMA.
bsl_status launch_compress24(const void *W, const bsl_semi24 *out, cudaStream_t s);
bsl_status launch_semi24_fwd(const void *X, int32_t M, const bsl_semi24 *W, const void *bias, void *Y,
                             cudaStream_t s);

// Block-sparse weight with 2:4 inside its blocks: compress the kept blocks,
// forward on the sparse MMA driven by the row-group plan.
bsl_status launch_bsr24_compress(const bsl_bsr *W, void *values24, uint16_t *meta24, cudaStream_t s);
bsl_status launch_bsr24_fwd(const void *X, int32_t M, const bsl_bsr *W, const void *values24,
                            const uint16_t *meta24, const void *bias, void *Y, cudaStream_t s);

// Expert (grouped) layer.  launch_grouped_rows: forward (A = X, out = Y) or,
// transposed, the input gradient (A = dY, out = dX).
bsl_status launch_grouped_rows(const void *A, int32_t T, const int32_t *offsets, const bsl_grouped *W, bool transposed,
                               const void *bias, void *out, int32_t zero_rest, cudaStream_t s);
bsl_status launch_grouped_dw(const void *dY, const void *X, int32_t T, const int32_t *offsets, const bsl_grouped *W,
                             void *dW, cudaStream_t s);
bsl_status launch_grouped_bias_grad(const void *dY, int32_t T, const int32_t *offsets, int32_t E, int32_t N, void *db,
                                    cudaStream_t s);

// The forwards of the layers for calls of few rows, where these are true.
bool few_rows(int32_t T, const bsl_grouped *W);
bool few_rows4(int32_t T, const bsl_mx4 *W);
bool few_rows8(int32_t T);
bsl_status launch_few_rows(const void *X, int32_t T, const int32_t *offsets, const bsl_grouped *W, const void *bias,
                           void *Y, int32_t zero_rest, cudaStream_t s);
bsl_status launch_few_rows4(const uint8_t *xc, const uint8_t *xs, int32_t T, const int32_t *offsets, const bsl_mx4 *W,
                            const void *bias, void *Y, int32_t zero_rest, cudaStream_t s);
bsl_status launch_few_rows8(const uint8_t *xc, const float *xs, int32_t T, const int32_t *offsets, const bsl_fp8 *W,
                            const void *bias, void *Y, int32_t zero_rest, cudaStream_t s);

// Microscaled 4-bit: conversion, and the product (offsets null: one group of all rows).
bsl_status launch_mx4_quantize(const void *X, int64_t elems, uint8_t *codes, uint8_t *scales, cudaStream_t s);
bsl_status launch_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t elems, void *X, cudaStream_t s);
bsl_status launch_mx4_fwd(const uint8_t *xc, const uint8_t *xs, int32_t T, const int32_t *offsets, const bsl_mx4 *W,
                          const void *bias, void *Y, int32_t zero_rest, cudaStream_t s);

// 8 bits with a scale for each block of 128: conversion, and the products (offsets null: one group of all rows;
// transposed: the input gradient; early: launched right behind the conversion of its rows, so that anything else that
// it reads is older than that kernel).
bsl_status launch_fp8_quantize(const void *X, int64_t planes, int64_t rows, int32_t K, bool tiles, uint8_t *codes,
                               float *scales, cudaStream_t s);
bsl_status launch_fp8_dequantize(const uint8_t *codes, const float *scales, int64_t planes, int64_t rows, int32_t K,
                                 bool tiles, void *X, cudaStream_t s);
bsl_status launch_fp8(const uint8_t *codes, const float *scales, int32_t T, const int32_t *offsets, const bsl_fp8 *W,
                      bool transposed, const void *bias, void *out, int32_t zero_rest, bool early, cudaStream_t s);
bool fp8_few(int32_t T, int32_t E, int32_t cols);
bsl_status launch_fp8_few(const uint8_t *codes, const float *scales, int32_t T, const int32_t *offsets, const bsl_fp8 *W,
                          bool transposed, const void *bias, void *out, int32_t zero_rest, bool early, cudaStream_t s);

// Router: choices, weights and (where order is not null) the pairs sorted by expert; the logits' gradient.
size_t route_workspace_bytes(int32_t T, int32_t E, int32_t k);
bsl_status launch_route(const void *logits, bool half, int32_t T, int32_t E, int32_t k, bool sigmoid, bool renormalize,
                        float factor, int32_t *experts, float *weights, int32_t *offsets, int32_t *order, void *workspace,
                        cudaStream_t s);
bsl_status launch_route_backward(const float *dweights, const void *logits, bool half, int32_t T, int32_t E, int32_t k,
                                 const int32_t *experts, bool sigmoid, bool renormalize, float factor, void *dlogits,
                                 cudaStream_t s);

// A whole expert layer for a few tokens; s13 and s2 null: bf16 weights, else 8 bits.
bsl_status launch_moe(const void *X, int32_t T, const int32_t *experts, const float *weights, int32_t k, const void *W13,
                      const float *s13, const void *W2, const float *s2, int32_t E, int32_t H, int32_t I, int32_t *status,
                      void *workspace, void *Y, cudaStream_t s);

bsl_status launch_debug_wait(int32_t *status, uint64_t timeout_ns, cudaStream_t s);

}  // namespace bsl
