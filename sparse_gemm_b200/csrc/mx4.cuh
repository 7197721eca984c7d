// mx4.cuh -- microscaled 4-bit codes to bf16 (mx4_quant.cu gives the format).
#pragma once

#include "common.cuh"

namespace bsl {

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Eight codes to four registers of two bf16: code j and code j + 4.  A code's
// bits s e e m, put at the sign, the lowest exponent bits and the highest
// mantissa bit of a bf16, are 2^-126 of its value, zero and 0.5 included, and
// one product brings 2^126 and the block's scale in.  Exact: two significant
// bits times a power of two.  The factor
// 2^126 x 2^(scale - 127) is past the bf16 range from scale byte 129 on: there
// it is brought in by two products, the second one `low` (a power of two, for
// values that are themselves past the range) smaller.
template <bool kHigh>
__device__ __forceinline__ void decode8(uint32_t w, uint32_t scale, uint32_t low, uint32_t (&v)[4])
{
    const uint32_t s1 = scale == 255 ? 0x7FC0u : scale > 128 ? 0x7F00u : scale ? (scale + 126u) << 7 : 0x3F00u;
    const uint32_t factor = s1 | s1 << 16;
    v[0] = (w << 12 & 0x80008000u) | (w << 6 & 0x01C001C0u);
    v[1] = (w << 8 & 0x80008000u) | (w << 2 & 0x01C001C0u);
    v[2] = (w << 4 & 0x80008000u) | (w >> 2 & 0x01C001C0u);
    v[3] = (w & 0x80008000u) | (w >> 6 & 0x01C001C0u);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = mul_bf16x2(v[i], factor);
    if (kHigh) {
        const uint32_t s2 = (scale > 128 && scale < 255 ? scale - 1u : 127u) - low;
        const uint32_t more = s2 << 7 | s2 << 23;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = mul_bf16x2(v[i], more);
    }
}

}  // namespace bsl
