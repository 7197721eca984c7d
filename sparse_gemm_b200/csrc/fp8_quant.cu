// fp8_quant.cu -- 8-bit floating point (e4m3) with a scale for each block of 128
// along K: bf16 to codes and scales, and back.  A block is 128 neighbours of one
// row (activations) or a tile of 128 rows by 128 columns (weights); the last
// ones of a row or column may be shorter.
//
// With a = max(largest magnitude of the block, 2^-100), each step in fp32:
//     s = a / 448      r = 448 / a      code = e4m3(x r), to nearest, ties to even
// 448 is the largest e4m3 number, and x r is at most 448 (1 + 2^-23), which
// rounds to it.  The bound on a keeps r finite; elements under such a scale are
// far below every bf16 product's last bit.  An infinity or NaN in the block
// makes its scale NaN and its codes zero, so all of it is NaN.
//
// Bound by bytes: 2 read and 1 written an element (the reverse back).  16 lanes
// read the 256 bytes of a row's block, and a thread has eight such loads in
// flight.  A CTA owns a tile, or as many elements of fewer and longer rows: up to
// eight blocks of a row side by side, 2 KB.
#include "common.cuh"
#include "internal.h"

namespace bsl {
namespace {

constexpr int kThreads = 256;

struct Fp8Args {
    const uint4 *X;
    uint2 *codes;
    float *scales;
    int64_t rows;  // of a plane
    int32_t K, kb, tiles;  // columns, blocks of a row, row tiles of a plane
    int32_t span;          // rows: log2 of the blocks of a row that a CTA takes
};

__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(lo), "f"(hi));
    return r;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Scale and factor of a block whose largest magnitude has the bf16 bits `top`.
__device__ __forceinline__ void scale_of(uint32_t top, float &s, float &r)
{
    const float a = fmaxf(__uint_as_float(top << 16), 0x1p-100f);
    s = __fdiv_rn(a, 448.f);
    r = __fdiv_rn(448.f, a);
    if (top >= 0x7F80u) {
        s = __uint_as_float(0x7FC00000u);
        r = 0.f;
    }
}

__device__ __forceinline__ uint32_t max16(uint32_t top, const uint4 &v)
{
    top = __vmaxu2(top, v.x & 0x7FFF7FFFu);
    top = __vmaxu2(top, v.y & 0x7FFF7FFFu);
    top = __vmaxu2(top, v.z & 0x7FFF7FFFu);
    return __vmaxu2(top, v.w & 0x7FFF7FFFu);
}

// Eight values to codes.  `some` is false where the block is not finite: x r would be NaN there.
__device__ __forceinline__ uint2 encode8(const uint4 &v, float r, bool some)
{
    if (!some) return make_uint2(0, 0);
    uint2 c;
    c.x = to_e4m3x2(bf16_lo(v.x) * r, bf16_hi(v.x) * r) | to_e4m3x2(bf16_lo(v.y) * r, bf16_hi(v.y) * r) << 16;
    c.y = to_e4m3x2(bf16_lo(v.z) * r, bf16_hi(v.z) * r) | to_e4m3x2(bf16_lo(v.w) * r, bf16_hi(v.w) * r) << 16;
    return c;
}

// A CTA's tile: plane, first row, block of the columns.
struct Where {
    int64_t plane, row0, left;
    int kt;
};

__device__ __forceinline__ Where tile_of(int64_t rows, int kb, int tiles)
{
    Where w;
    const uint32_t t = blockIdx.x / static_cast<uint32_t>(kb);
    w.kt = static_cast<int>(blockIdx.x - t * static_cast<uint32_t>(kb));
    const uint32_t p = t / static_cast<uint32_t>(tiles);
    w.plane = p;
    w.row0 = static_cast<int64_t>(t - p * static_cast<uint32_t>(tiles)) * 128;
    w.left = rows - w.row0;
    return w;
}

// Rows: 16 lanes a block, a CTA 2^span blocks of 128 >> span rows, a thread eight
// rows.  The eight maxima over 16 lanes take eight shuffles: in each step a lane
// keeps half of its rows and gives the other half away, so that lane l ends up
// with row l & 7 (of its half of the lanes, and one more step), divides for it alone,
// and hands the factor out.  (A reduction and two divisions a row and lane: twice the
// instructions, 26 us instead of 17 at 8192 x 4096.)
__global__ void __launch_bounds__(kThreads) k_fp8_quantize_rows(const Fp8Args a)
{
    const int lane = threadIdx.x & 15, group = threadIdx.x >> 4, span = a.span;
    const uint32_t wide = (static_cast<uint32_t>(a.kb) + (1u << span) - 1) >> span;
    const uint32_t t = blockIdx.x / wide;
    const int b = static_cast<int>(blockIdx.x - t * wide) << span | (group & ((1 << span) - 1));
    const int64_t row0 = static_cast<int64_t>(t) * (128 >> span) + (group >> span);
    const int step = 16 >> span, col = b * 128 + 8 * lane;
    const int rows = static_cast<int>(a.rows - row0 < 128 ? a.rows - row0 : 128);  // of this thread: i step < rows
    const int64_t first = (row0 * a.K + col) / 8;
    const int64_t stride = static_cast<int64_t>(step) * a.K / 8;
    const bool in = col < a.K;
    wait_for_prior_grid();
    // behind the wait: the product that follows reads weights and offsets before its own wait
    dependents_may_launch();
    uint4 x[8];
    uint32_t top[8];
    const uint4 *from = a.X + first;
#pragma unroll
    for (int i = 0; i < 8; ++i, from += stride) {
        x[i] = make_uint4(0, 0, 0, 0);
        if (in && i * step < rows) x[i] = load_stream(from);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        top[i] = max16(0, x[i]);
        top[i] = max(top[i] & 0xFFFFu, top[i] >> 16);
    }
#pragma unroll
    for (int d = 4; d; d >>= 1) {
        const bool upper = lane & d;
#pragma unroll
        for (int i = 0; i < d; ++i) {
            const uint32_t give = upper ? top[i] : top[i + d], keep = upper ? top[i + d] : top[i];
            top[i] = max(keep, __shfl_xor_sync(0xffffffffu, give, d));
        }
    }
    top[0] = max(top[0], __shfl_xor_sync(0xffffffffu, top[0], 8));  // of row lane & 7
    float s, f;
    scale_of(top[0], s, f);
    const int mine = (lane & 7) * step;
    if (lane < 8 && mine < rows && b < a.kb) a.scales[(row0 + mine) * a.kb + b] = s;
    uint2 *to = a.codes + first;
#pragma unroll
    for (int i = 0; i < 8; ++i, to += stride) {
        const float r = __shfl_sync(0xffffffffu, f, i, 16);  // 0 where the block is not finite
        if (in && i * step < rows) *to = encode8(x[i], r, r != 0.f);
    }
}

__global__ void __launch_bounds__(kThreads) k_fp8_quantize_tiles(const Fp8Args a)
{
    __shared__ uint32_t tops[kThreads / 32];
    const Where w = tile_of(a.rows, a.kb, a.tiles);
    const int lane = threadIdx.x & 15, group = threadIdx.x >> 4;
    const int col = w.kt * 128 + 8 * lane;
    const int64_t first = w.plane * a.rows + w.row0;
    dependents_may_launch();
    wait_for_prior_grid();
    uint4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = group + 16 * i;
        x[i] = make_uint4(0, 0, 0, 0);
        if (r < w.left && col < a.K) x[i] = load_stream(a.X + ((first + r) * a.K + col) / 8);
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max16(top, x[i]);
    top = max(top & 0xFFFFu, top >> 16);
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) top = max(top, tops[i]);
    float s, f;
    scale_of(top, s, f);
    if (threadIdx.x == 0) a.scales[blockIdx.x] = s;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = group + 16 * i;
        if (row < w.left && col < a.K) a.codes[((first + row) * a.K + col) / 8] = encode8(x[i], f, top < 0x7F80u);
    }
}

// Two codes to their values, exact.
__device__ __forceinline__ float2 from_e4m3x2(uint32_t two)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
    float2 f;
    asm("{\n\t.reg .f16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(h));
    return f;
}

__device__ __forceinline__ uint4 decode8(uint32_t lo, uint32_t hi, float s)
{
    const float2 a = from_e4m3x2(lo & 0xFFFFu), b = from_e4m3x2(lo >> 16);
    const float2 c = from_e4m3x2(hi & 0xFFFFu), d = from_e4m3x2(hi >> 16);
    return make_uint4(pack_bf16x2(a.x * s, a.y * s), pack_bf16x2(b.x * s, b.y * s), pack_bf16x2(c.x * s, c.y * s),
                      pack_bf16x2(d.x * s, d.y * s));
}

template <bool kTiles>
__global__ void __launch_bounds__(kThreads)
    k_fp8_dequantize(const uint2 *codes, const float *scales, int64_t rows, int32_t K, int32_t kb, int32_t tiles, uint4 *X)
{
    const Where w = tile_of(rows, kb, tiles);
    const int lane = threadIdx.x & 15, group = threadIdx.x >> 4;
    const int col = w.kt * 128 + 8 * lane, left = static_cast<int>(w.left < 128 ? w.left : 128);
    const int64_t row0 = w.plane * rows + w.row0 + group, first = (row0 * K + col) / 8, stride = 2ll * K;
    const bool in = col < K;
    dependents_may_launch();
    wait_for_prior_grid();
    uint2 c[8];
    float s[8];
    if (kTiles) s[0] = load_float(scales + blockIdx.x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        c[i] = make_uint2(0, 0);
        if (!kTiles) s[i] = 0.f;
        if (in && group + 16 * i < left) {
            c[i] = load_global(codes + first + i * stride);
            if (!kTiles) s[i] = load_float(scales + (row0 + 16 * i) * kb + w.kt);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (in && group + 16 * i < left) X[first + i * stride] = decode8(c[i].x, c[i].y, s[kTiles ? 0 : i]);
}

// CTAs of a conversion, 0 if they are too many.
unsigned tile_count(int64_t planes, int64_t rows, int32_t K)
{
    const int64_t per = (rows + 127) / 128 * ((K + 127) / 128);
    return planes > 0x7FFFFFFF / per ? 0 : static_cast<unsigned>(planes * per);
}

}  // namespace

bsl_status launch_fp8_quantize(const void *X, int64_t planes, int64_t rows, int32_t K, bool tiles, uint8_t *codes,
                               float *scales, cudaStream_t s)
{
    Fp8Args a = {static_cast<const uint4 *>(X), reinterpret_cast<uint2 *>(codes), scales, rows, K, (K + 127) / 128, 0, 0};
    if (tiles) {
        const unsigned grid = tile_count(planes, rows, K);
        if (!grid) return BSL_ERR_UNSUPPORTED;
        a.tiles = static_cast<int32_t>((rows + 127) / 128);
        return cuda_status(launch_dependent(k_fp8_quantize_tiles, grid, kThreads, 0, s, a));
    }
    a.rows = planes * rows;
    while (a.span < 3 && (2 << a.span) <= a.kb) ++a.span;
    const int64_t wide = (a.kb + (1 << a.span) - 1) >> a.span, high = (a.rows + (128 >> a.span) - 1) / (128 >> a.span);
    if (high > 0x7FFFFFFF / wide) return BSL_ERR_UNSUPPORTED;
    return cuda_status(launch_dependent(k_fp8_quantize_rows, static_cast<unsigned>(wide * high), kThreads, 0, s, a));
}

bsl_status launch_fp8_dequantize(const uint8_t *codes, const float *scales, int64_t planes, int64_t rows, int32_t K,
                                 bool tiles, void *X, cudaStream_t s)
{
    const unsigned grid = tile_count(planes, rows, K);
    if (!grid) return BSL_ERR_UNSUPPORTED;
    return cuda_status(launch_dependent(tiles ? k_fp8_dequantize<true> : k_fp8_dequantize<false>, grid, kThreads, 0, s,
                                        reinterpret_cast<const uint2 *>(codes), scales, rows, K, (K + 127) / 128,
                                        static_cast<int32_t>((rows + 127) / 128), static_cast<uint4 *>(X)));
}

}  // namespace bsl
