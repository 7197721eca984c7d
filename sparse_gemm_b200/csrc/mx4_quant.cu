// mx4_quant.cu -- microscaled 4-bit floating point (OCP MX, "MXFP4"): bf16 to
// 4-bit codes with one power-of-two scale for 32 neighbours along K, and back.
//
// For a block of 32 with largest magnitude a (finite):
//     s = 2^(max(floor(log2 a), -125) - 2)        scale byte = log2 s + 127
//     q = x / s to the nearest of 0 .5 1 1.5 2 3 4 6 (ties to the even code), 6 at most
// floor(log2 a) is the exponent field f of a's bf16 bits less 127, so the
// scale byte is max(f - 2, 0); x / s is a product with a power of two, exact
// in fp32, so the one rounding is the conversion to 4 bits.  f = 255 (an
// infinity or NaN in the block) gives the scale byte 255, which stands for
// NaN, and zero codes.
//
// Bound by bytes: 2 read and 17/32 written an element (the reverse back).
// Four lanes share a block: 16-byte loads, 4-byte code stores, whole lines a
// warp; the largest magnitude takes two shuffles.  A thread has kChunks such
// loads in flight, a block's width apart.
#include "common.cuh"
#include "internal.h"

namespace bsl {
namespace {

constexpr int kThreads = 256;
constexpr int kChunks = 4;  // a thread's chunks of 8 elements

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two values to two 4-bit codes, `lo` in the low half.
__device__ __forceinline__ uint32_t to_e2m1x2(float lo, float hi)
{
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\t"
        "cvt.u32.u8 %0, b;\n\t}"
        : "=r"(r)
        : "f"(lo), "f"(hi));
    return r;
}

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
// bits times a power of two.  The factor 2^126 x 2^(scale - 127) is past the
// bf16 range from scale byte 129 on: there two products bring it in.
__device__ __forceinline__ void decode8(uint32_t w, uint32_t scale, uint32_t (&v)[4])
{
    const uint32_t s1 = scale == 255 ? 0x7FC0u : scale > 128 ? 0x7F00u : scale ? (scale + 126u) << 7 : 0x3F00u;
    const uint32_t s2 = (scale > 128 && scale < 255 ? scale - 1u : 127u) << 7;
    v[0] = (w << 12 & 0x80008000u) | (w << 6 & 0x01C001C0u);
    v[1] = (w << 8 & 0x80008000u) | (w << 2 & 0x01C001C0u);
    v[2] = (w << 4 & 0x80008000u) | (w >> 2 & 0x01C001C0u);
    v[3] = (w & 0x80008000u) | (w >> 6 & 0x01C001C0u);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = mul_bf16x2(mul_bf16x2(v[i], s1 | s1 << 16), s2 | s2 << 16);
}

// Chunk i covers elements 8i .. 8i+7; n is the number of chunks, a multiple of 4.
__global__ void __launch_bounds__(kThreads)
    k_mx4_quantize(const uint4 *X, int64_t n, uint32_t *codes, uint8_t *scales)
{
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kThreads * kChunks + threadIdx.x;
    dependents_may_launch();
    wait_for_prior_grid();
    uint4 x[kChunks];
#pragma unroll
    for (int u = 0; u < kChunks; ++u) {
        const int64_t i = i0 + u * kThreads;
        x[u] = i < n ? load_global(X + i) : make_uint4(0, 0, 0, 0);  // a block's four lanes are in or out together
    }
#pragma unroll
    for (int u = 0; u < kChunks; ++u) {
        const int64_t i = i0 + u * kThreads;
        const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) top = __vmaxu2(top, w[j] & 0x7FFF7FFFu);
        top = max(top & 0xFFFFu, top >> 16);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const uint32_t f = top >> 7;
        const uint32_t scale = f == 255 ? 255 : f > 2 ? f - 2 : 0;
        // 1 / s = 2^(127 - scale)
        const float inv = __uint_as_float((254 - scale) << 23);
        uint32_t code = 0;
        if (f != 255) {
#pragma unroll
            for (int j = 0; j < 4; ++j) code |= to_e2m1x2(bf16_lo(w[j]) * inv, bf16_hi(w[j]) * inv) << (8 * j);
        }
        if (i >= n) continue;
        codes[i] = code;
        if ((i & 3) == 0) scales[i >> 2] = static_cast<uint8_t>(scale);
    }
}

__global__ void __launch_bounds__(kThreads)
    k_mx4_dequantize(const uint32_t *codes, const uint8_t *scales, int64_t n, uint4 *X)
{
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kThreads * kChunks + threadIdx.x;
    dependents_may_launch();
    wait_for_prior_grid();
    uint32_t c[kChunks], b[kChunks];
#pragma unroll
    for (int u = 0; u < kChunks; ++u) {
        const int64_t i = i0 + u * kThreads;
        c[u] = i < n ? load_global(codes + i) : 0;
        b[u] = i < n ? load_global(scales + (i >> 2)) : 0;
    }
#pragma unroll
    for (int u = 0; u < kChunks; ++u) {
        const int64_t i = i0 + u * kThreads;
        uint32_t v[4];  // codes j and j + 4
        decode8(c[u], b[u], v);
        if (i < n)
            X[i] = make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410),
                              __byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632));
    }
}

}  // namespace

bsl_status launch_mx4_quantize(const void *X, int64_t elems, uint8_t *codes, uint8_t *scales, cudaStream_t s)
{
    const int64_t n = elems / 8, blocks = (n + kThreads * kChunks - 1) / (kThreads * kChunks);
    if (blocks > 0x7FFFFFFF) return BSL_ERR_UNSUPPORTED;
    return cuda_status(launch_dependent(k_mx4_quantize, static_cast<unsigned>(blocks), kThreads, 0, s,
                                        static_cast<const uint4 *>(X), n, reinterpret_cast<uint32_t *>(codes), scales));
}

bsl_status launch_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t elems, void *X, cudaStream_t s)
{
    const int64_t n = elems / 8, blocks = (n + kThreads * kChunks - 1) / (kThreads * kChunks);
    if (blocks > 0x7FFFFFFF) return BSL_ERR_UNSUPPORTED;
    return cuda_status(launch_dependent(k_mx4_dequantize, static_cast<unsigned>(blocks), kThreads, 0, s,
                                        reinterpret_cast<const uint32_t *>(codes), scales, n, static_cast<uint4 *>(X)));
}

}  // namespace bsl
