// grouped.cuh -- the row ranges of the experts, as every grouped kernel reads them.
#pragma once

#include "common.cuh"

namespace bsl {

constexpr int kMaxExperts = BSL_GROUPED_MAX_EXPERTS;

// Copy offsets[0..E] into shared memory, made safe by the first warp: every
// entry is clamped to [previous entry, T], so no value on the device can lead
// outside the matrices; one that had to be clamped is reported in `status`.
// The caller synchronises the block before reading off[].
__device__ __forceinline__ void load_offsets(const int32_t *offsets, int32_t E, int32_t T, int32_t *off,
                                             int32_t *status)
{
    if (threadIdx.x >= 32) return;
    const int lane = threadIdx.x;
    int carry = 0;
    bool bad = false;
    for (int i0 = 0; i0 <= E; i0 += 32) {
        const int i = i0 + lane;
        const int raw = i <= E ? offsets[i] : 0;
        int v = raw < 0 ? 0 : raw > T ? T : raw;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, v, d);
            if (lane >= d && o > v) v = o;
        }
        if (v < carry) v = carry;
        if (i <= E) {
            off[i] = v;
            bad |= v != raw;
        }
        carry = __shfl_sync(0xffffffffu, v, 31);
    }
    if (bad) set_status(status, BSL_ERR_INVALID_ARG);
}

}  // namespace bsl
