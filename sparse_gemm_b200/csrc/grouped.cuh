// grouped.cuh -- what the grouped kernels share: the row ranges of the experts
// and the list of output tiles over them.
#pragma once

#include "common.cuh"
#include "pair.cuh"

namespace bsl {

constexpr int kMaxExperts = BSL_GROUPED_MAX_EXPERTS;

// The experts' offsets[0..E] into shared memory, by the whole block (which
// synchronises before clamp_offsets).  offsets null: one expert (E = 1) owns
// all rows.
__device__ __forceinline__ void fetch_offsets(const int32_t *offsets, int32_t E, int32_t T, int32_t *off)
{
    for (int i = threadIdx.x; i <= E; i += blockDim.x) off[i] = offsets ? load_global(offsets + i) : i ? T : 0;
}

// Make them safe, by one warp: every entry is clamped to [previous entry, T],
// so no value on the device can lead outside the matrices; one that had to be
// clamped is reported in `status`.  The block synchronises before it uses them.
__device__ __forceinline__ void clamp_offsets(int32_t E, int32_t T, int32_t *off, int32_t *status)
{
    const int lane = threadIdx.x & 31;
    int carry = 0;
    bool bad = false;
    for (int i0 = 0; i0 <= E; i0 += 32) {
        const int i = i0 + lane;
        const int raw = i <= E ? off[i] : 0;
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
    __syncwarp();
}

// Row tile i when `rows` rows are cut into the fewest tiles of at most `most`
// rows: their units of `step` rows (most is a multiple of step) are spread
// evenly, so tiles differ by one unit and only the last one holds rows that do
// not exist, fewer than a unit.
__device__ __forceinline__ void row_tile(int rows, int most, int step, int i, int &first, int &n)
{
    const int tiles = (rows + most - 1) / most, units = (rows + step - 1) / step;
    const int q = units / tiles, more = units - q * tiles;
    first = (i * q + (i < more ? i : more)) * step;
    n = (q + (i < more)) * step;
}

// Prefix sums by the calling warp: start[i] = sum of count(j) over j < i, i = 0 .. E.
template <typename Count>
__device__ __forceinline__ void tile_starts(int32_t E, int32_t *start, Count count)
{
    const int lane = threadIdx.x & 31;
    int carry = 0;
    for (int i0 = 0; i0 < E; i0 += 32) {
        const int i = i0 + lane;
        const int c = i < E ? count(i) : 0;
        int v = c;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, v, d);
            if (lane >= d) v += o;
        }
        if (i < E) start[i] = carry + v - c;
        carry += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) start[E] = carry;
    __syncwarp();
}

// Expert of tile t (start[0] <= t < start[E]): the last i with start[i] <= t.
__device__ __forceinline__ int expert_of(const int32_t *start, int32_t E, int t)
{
    int lo = 0, hi = E - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Row and column tile of tile i of one expert's nr x nc: bands of kBand row
// tiles, column tile major inside a band, so that tiles taken at one time
// share few weight tiles and one band of rows, both in L2.
constexpr int kBand = 8;

__device__ __forceinline__ void tile_place(int i, int nr, int nc, int &r, int &c)
{
    const int band = i / (kBand * nc), in = i - band * kBand * nc, first = band * kBand;
    const int width = nr - first < kBand ? nr - first : kBand;
    c = in / width;
    r = first + in - c * width;
}

// Zero out[a .. b) (elements, multiples of 8) with one warp of every CTA.
__device__ __forceinline__ void zero_range(__nv_bfloat16 *out, int64_t a, int64_t b, int lane)
{
    uint4 *p = reinterpret_cast<uint4 *>(out);
    for (int64_t i = a / 8 + static_cast<int64_t>(blockIdx.x) * 32 + lane; i < b / 8;
         i += static_cast<int64_t>(gridDim.x) * 32)
        p[i] = make_uint4(0, 0, 0, 0);
}

// One warp's 32 x 32 part of an accumulator: lane = output column, v[i] = row i
// (fp32 bits), to bf16 rows of 64 bytes in shared memory.  Neighbouring lanes
// swap halves, so each writes whole words (two columns of one row); a warp's
// store covers 128 contiguous bytes.
__device__ __forceinline__ void stage_chunk(uint8_t *dst, const uint32_t (&v)[32], float bias, int lane)
{
    const uint32_t odd = lane & 1;
    const uint32_t sel = odd ? 0x3276u : 0x5410u;  // odd: (other.hi, own.hi); even: (own.lo, other.lo)
#pragma unroll
    for (int u = 0; u < 16; ++u) {
        const uint32_t own = pack_bf16x2(__uint_as_float(v[2 * u]) + bias, __uint_as_float(v[2 * u + 1]) + bias);
        const uint32_t other = __shfl_xor_sync(0xffffffffu, own, 1);
        *reinterpret_cast<uint32_t *>(dst + (2 * u + odd) * 64 + (lane & ~1) * 2) = __byte_perm(own, other, sel);
    }
}

// Rows 0 .. rows-1 of a staged chunk to global memory, 16 bytes a lane:
// `out` points at the chunk's first element, `left` columns exist (a multiple of 8).
__device__ __forceinline__ void store_rows(__nv_bfloat16 *out, int64_t stride, const uint8_t *src, int rows, int left,
                                           int lane)
{
    const int part = lane & 3;
    for (int r = lane >> 2; r < rows; r += 8)
        if (8 * part < left)
            *reinterpret_cast<uint4 *>(out + r * stride + 8 * part) =
                *reinterpret_cast<const uint4 *>(src + r * 64 + 16 * part);
}

}  // namespace bsl
