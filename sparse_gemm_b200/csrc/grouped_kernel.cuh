// grouped_kernel.cuh -- the tensor-core kernel of the expert (grouped) layer, for
// bf16 and for microscaled 4-bit operands.
//
// The rows of X are sorted by expert: rows offsets[e] .. offsets[e+1] - 1 are
// multiplied with expert e's weight W[e] [N][K]:
//     forward          Y[t]  = X[t] . W[e]^T + bias[e]
//     input gradient   dX[t] = dY[t] . W[e]
//     weight gradient  dW[e] = sum over the rows t of e of dY[t]^T . X[t]
// (bf16 in, fp32 accumulation in TMEM, one rounding to bf16).
//
// One kernel for the three.  Each is, for an expert, out[r][c] = sum_k A(c, k)
// B(r, k), and out's contiguous index c (features) goes to the MMA's M side,
// i.e. to the TMEM lanes, its row index r to the N side:
//                      A (c, k)            B (r, k)          ragged
//     forward          W[e]   K-major      X     K-major     r
//     input gradient   W[e]^T M-major      dY    K-major     r
//     weight gradient  X^T    M-major      dY^T  N-major     k
// The MMA's N may be any multiple of 16, so a tile with few rows costs few
// rows: an expert's rows are spread evenly over the fewest tiles of 256.  Rows of
// the next expert that a copy brings along only reach accumulator columns
// that are never stored.  For the weight gradient, whose ragged index is
// summed over, k_expert_maps first writes a tensor map for each expert's rows,
// and the copies fill the rows behind its last one with zeros (a NaN there
// must not meet a zero).
//
// Persistent kernels, programmatic dependents, 8 warps a CTA:
//   warps 0, 2 TMA producers of A and of B (a ring of stages);
//   warp 1     MMA issuer and TMEM owner;
//   warp 3     zeros for the rows of no expert, on request;
//   warps 4-7  epilogue: TMEM -> registers (+ bias) -> bf16, transposed
//              through 2 KB of shared memory, TMA store of 32 x 32 chunks;
//              chunks that end inside an expert's rows with plain stores.
// Two accumulators: a tile's epilogue overlaps the next tile's MMAs.  Tiles
// are dealt round robin; no counters and no workspace are shared by calls,
// and every output is one sum in a fixed order.
//
// kPair: clusters of two CTAs on tiles of 256 features x 256 rows
// (cta_group::2, M = 256; each CTA holds its 128 rows of A and half of B),
// three stages of 128 k.  Bound by the tensor pipe only while the copies keep
// up (32 KB per 64 k and SM, 64 bytes a clock), and those go by their number:
// an operand's stage is one copy of 32 KB, two strips of 128-byte rows.  At
// 16384 x 4096 x 14336, 8 experts, kernels back to back (clock held by power
// at 1.1-1.3 GHz): one 32 KB copy 1412 / 1459 / 1460 us for the three, copies
// of 16 KB and stages of 64 k 1460 / 1575 / 1540, of 8 KB (gradients) 1775.
//
// Otherwise (forward with few rows, which reads each weight once): one CTA on
// `h` = 128, 64 or 32 features x 64, 32 or 16 rows; a stage always holds
// 16 KB of the weight, i.e. 64, 128 or 256 k, so small h only spreads the same
// stream over more SMs.  The MMA still takes 128 rows of A; those past h are
// other bytes of the ring and reach lanes that are never stored.
//
// Every wait is bounded (BSL_ERR_TIMEOUT in the status word, then all roles
// leave through an abort flag).
#pragma once

#include "common.cuh"
#include "grouped.cuh"
#include "internal.h"

namespace bsl {
namespace {

enum Mode { kForward = 0, kInputGrad = 1, kWeightGrad = 2, kForward4 = 3, kForward4Any = 4 };
// kForward4: rows of scales in whole 16-byte units (K a multiple of 512); kForward4Any: any K

template <int kMode, bool kPair>
struct Cfg {
    static constexpr bool F4 = kMode == kForward4 || kMode == kForward4Any;
    static constexpr int CG = kPair ? 2 : 1;
    static constexpr int BR = kPair ? (F4 ? 224 : 256) : 64;  // rows per tile, at most (h = 128)
    static constexpr int STEP = 16 * CG;                 // granularity of the rows (MMA N)
    static constexpr int BOX = 16;                       // rows of B's smallest copy box
    static constexpr int BK = kPair ? 128 : 64;          // k per stage (h = 128)
    static constexpr int A_BYTES = 128 * BK * 2;
    static constexpr int B_BYTES = BR / CG * BK * 2;
    // scales of a stage: chunks of 512 bytes for 128 rows x 128 elements
    static constexpr int SA_BYTES = !F4 ? 0 : kPair ? 4 * 512 : 8 * 512;
    static constexpr int SB_BYTES = !F4 ? 0 : 8 * 512;
    static constexpr int STAGE = A_BYTES + B_BYTES + SA_BYTES + SB_BYTES;
    static constexpr int S = kPair ? 3 : 196608 / STAGE; // otherwise 8 stages, 6 with scales
    // two accumulators, then the scales of the stage at work (A 4, B 4 or 8 columns a chunk)
    static constexpr int SA_COL = 2 * BR, SB_COL = SA_COL + SA_BYTES / 128;
    static constexpr int TMEM = !F4 ? 2 * BR : kPair ? 512 : 256;
    static constexpr int CHUNK = 32 * 32 * 2;
    static constexpr int OUT = 4 * 2 * CHUNK;            // two chunks per epilogue warp
    static constexpr int BARS = (2 * S + 5) * 8 + 16;
    static constexpr int SMEM = 1024 + S * STAGE + OUT + BARS + 2 * (kMaxExperts + 1) * 4;
    static constexpr int SCALE_WARPS = !F4 ? 0 : kPair ? 3 : 2;  // of a stage
    static constexpr int SCALE_SETS = 2;                         // taking stages in turn
    static constexpr int THREADS = 256 + 32 * SCALE_WARPS * SCALE_SETS;
    static_assert(SMEM <= 227 * 1024, "shared memory");
    static_assert(STAGE % 1024 == 0, "swizzle atoms");
    static_assert(!F4 || SB_COL + SB_BYTES / 128 <= TMEM, "TMEM columns");
};

struct Maps {
    // pair: a[0] two strips a copy, a[1] one strip; b[i] two strips of 16 (i + 1) rows, b[8] one of 16 rows
    // otherwise: a[0..2] K-major boxes of 128, 64, 32 features; b[8] of 16 rows
    CUtensorMap a[3], b[9], out;
};

struct Args {
    const int32_t *offsets;
    const __nv_bfloat16 *bias;
    __nv_bfloat16 *out;
    const CUtensorMap *expert_maps;  // weight gradient: [E][4], see k_expert_maps
    int32_t *status;
    int32_t T, E;
    int32_t cols, rows, depth;       // of the product; the ragged one is unused
    int32_t zero_rest;
    const uint8_t *a_scales, *b_scales;  // 4-bit forward: [E][cols][scale_bytes], [T][scale_bytes]
    int32_t scale_bytes;
    uint64_t timeout_ns;
};

struct Tile {
    int e, c0;        // expert, first column
    int r0;           // first row: of the matrix, or of the expert's dW
    int n, valid;     // MMA N, rows that exist
    int k, kb;        // length of the sums, stages
};

// The tile list of a launch, the same in every CTA.
template <int kMode, bool kPair>
struct Tiles {
    const int32_t *off, *start;
    int E, h, cols, rows, depth;

    __device__ __forceinline__ int features() const { return kPair ? 256 : h; }
    __device__ __forceinline__ int most() const { return kPair ? Cfg<kMode, kPair>::BR : h / 2; }
    __device__ __forceinline__ int stage_k() const { return kPair ? 128 : 64 * (128 / h); }
    __device__ __forceinline__ int count() const { return start[E]; }

    __device__ __forceinline__ Tile at(int t) const
    {
        Tile x;
        x.e = expert_of(start, E, t);
        const int first = off[x.e], own = off[x.e + 1] - first;
        const int r = kMode == kWeightGrad ? rows : own;
        constexpr int step = Cfg<kMode, kPair>::STEP;
        int ri, ci, r0;
        tile_place(t - start[x.e], (r + most() - 1) / most(), (cols + features() - 1) / features(), ri, ci);
        x.c0 = ci * features();
        if (kMode == kWeightGrad) {  // whole strips: full tiles and a shorter last one
            r0 = ri * most();
            x.n = r - r0 < most() ? (r - r0 + step - 1) / step * step : most();
        } else {
            row_tile(r, most(), step, ri, r0, x.n);
        }
        x.valid = r - r0 < x.n ? r - r0 : x.n;
        x.r0 = kMode == kWeightGrad ? r0 : first + r0;
        x.k = kMode == kWeightGrad ? own : depth;
        x.kb = (x.k + stage_k() - 1) / stage_k();
        return x;
    }
};

__device__ __forceinline__ uint8_t *align1024(uint8_t *p)
{
    return reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

// Features of a tile of the unpaired kernel.  Halving h keeps the SMs evenly
// loaded when there are few tiles, as long as no expert's rows need a second
// tile (which would read the weight twice).  Cost: rounds of tiles times the
// weight rows of one, plus 16 for what a tile costs besides.
__device__ __forceinline__ int pick_h(const int32_t *off, int E, int cols)
{
    const int lane = threadIdx.x & 31;
    int live[3] = {0, 0, 0}, top = 0;
    for (int e = lane; e < E; e += 32) {
        const int r = off[e + 1] - off[e];
        top = max(top, r);
#pragma unroll
        for (int i = 0; i < 3; ++i) live[i] += (r + (64 >> i) - 1) / (64 >> i);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    int best = 128;
    int64_t cost = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const int h = 128 >> i;
        const int64_t tiles = static_cast<int64_t>(__reduce_add_sync(0xffffffffu, live[i])) * ((cols + h - 1) / h);
        const int64_t c = (tiles + gridDim.x - 1) / gridDim.x * (h + 16);
        if (i == 0 || (top <= (64 >> i) && c < cost)) {
            best = h;
            cost = c;
        }
    }
    return best;
}

// ------------------------------------------------------------ scales (4-bit forward)
//
// The block-scaled MMA takes its scales from TMEM: row r of 128 has, for 128
// elements of k (four blocks of 32), four bytes at lane r % 32, column r / 32,
// the same in all four quarters of the lanes.  A chunk in shared memory is
// that arrangement as 32 rows of 16 bytes, which one tcgen05.cp spreads.  The
// scales lie in plain rows in global memory, wherever an expert's rows begin,
// so warps load each row's bytes (ahead, in registers) and write the chunks.

// Loads must not wait for one another, so nothing is computed on what was
// loaded before it is stored.  Bytes past the row's end count as zeros (a
// scale of 2^-127 on zero codes; a NaN byte of the next row must not reach
// them), and so do rows that do not exist.

// Whole rows of 16-byte units: W words of a row from byte0 on.
template <int W>
__device__ __forceinline__ void load_words(const uint8_t *base, int32_t stride, int64_t row, bool exists, int32_t byte0,
                                           uint32_t *w)
{
    constexpr int V = W < 4 ? W : 4;
    const uint8_t *at = base + row * stride + byte0;
#pragma unroll
    for (int i = 0; i < W; i += V) {
        const bool in = exists && byte0 + 4 * i < stride;
        if constexpr (V == 4) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (in) v = __ldg(reinterpret_cast<const uint4 *>(at + 4 * i));
            w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
        } else {
            uint2 v = make_uint2(0, 0);
            if (in) v = __ldg(reinterpret_cast<const uint2 *>(at + 4 * i));
            w[i] = v.x, w[i + 1] = v.y;
        }
    }
}

// Rows that start at any byte: the W + 1 aligned words around them, as far as
// they lie inside the `total` bytes ...
template <int W>
__device__ __forceinline__ void load_words_any(const uint8_t *base, int64_t total, int32_t stride, int64_t row, bool exists,
                                               int32_t byte0, uint32_t *w)
{
    const int64_t at = (row * stride + byte0) & ~int64_t(3);
#pragma unroll
    for (int i = 0; i <= W; ++i) {
        w[i] = 0;
        if (exists && at + 4 * i + 4 <= total) w[i] = __ldg(reinterpret_cast<const uint32_t *>(base + at + 4 * i));
    }
}

// ... and, when they are stored, shifted into place and cut at the row's end.
// The last bytes of the array may fill no whole word: they are read here.
template <int W>
__device__ __forceinline__ void shift_words(const uint8_t *base, int64_t total, int32_t stride, int64_t row, bool exists,
                                            int32_t byte0, const uint32_t *raw, uint32_t *w)
{
    const int64_t at = row * stride + byte0, low = at & ~int64_t(3);
    const int32_t left = exists ? stride - byte0 : 0;
    const uint32_t shift = static_cast<uint32_t>(at & 3) * 8;
    uint32_t r[W + 1];
#pragma unroll
    for (int i = 0; i <= W; ++i) {
        r[i] = raw[i];
        const int64_t a = low + 4 * i;
        if (exists && a < total && a + 4 > total)
            for (int b = 0; a + b < total; ++b) r[i] |= static_cast<uint32_t>(base[a + b]) << (8 * b);
    }
#pragma unroll
    for (int i = 0; i < W; ++i) {
        const int32_t bytes = left - 4 * i;
        const uint32_t v = __funnelshift_r(r[i], r[i + 1], shift);
        w[i] = bytes >= 4 ? v : bytes <= 0 ? 0 : v & ((1u << (8 * bytes)) - 1u);
    }
}

// Where a lane finds its rows of a stage: row, row + 32, ... of which `live` exist from `row` on.
struct ScaleRows {
    const uint8_t *base;
    int64_t total, row;
    int32_t stride, live, byte0;
};

// One warp's part of a stage: R rows a lane, W words each (W + 1 as loaded, for any K).
template <bool kAny, int R, int W>
__device__ __forceinline__ void load_scales(const ScaleRows &s, uint32_t *w)
{
#pragma unroll
    for (int c = 0; c < R; ++c) {
        if constexpr (kAny)
            load_words_any<W>(s.base, s.total, s.stride, s.row + 32 * c, 32 * c < s.live, s.byte0, w + c * (W + 1));
        else
            load_words<W>(s.base, s.stride, s.row + 32 * c, 32 * c < s.live, s.byte0, w + c * W);
    }
}

// Chunk j of the stage holds word j of every row: 16 bytes a lane.
template <bool kAny, int R, int W>
__device__ __forceinline__ void store_scales(uint8_t *dst, int step, int lane, const ScaleRows &s, const uint32_t *raw)
{
    uint32_t w[4][W];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        if (c >= R) {
#pragma unroll
            for (int j = 0; j < W; ++j) w[c][j] = 0;
        } else if constexpr (kAny) {
            shift_words<W>(s.base, s.total, s.stride, s.row + 32 * c, 32 * c < s.live, s.byte0, raw + c * (W + 1), w[c]);
        } else {
#pragma unroll
            for (int j = 0; j < W; ++j) w[c][j] = raw[c * W + j];
        }
    }
#pragma unroll
    for (int j = 0; j < W; ++j)
        *reinterpret_cast<uint4 *>(dst + j * step + lane * 16) = make_uint4(w[0][j], w[1][j], w[2][j], w[3][j]);
}

// A walk over this CTA's stages, tile after tile.
template <int kMode, bool kPair>
struct Walk {
    const Tiles<kMode, kPair> &tiles;
    int t, stride, count, k;
    Tile x;

    __device__ __forceinline__ Walk(const Tiles<kMode, kPair> &l, int first, int step, int n)
        : tiles(l), t(first), stride(step), count(n), k(0)
    {
        if (t < count) x = tiles.at(t);
    }
    __device__ __forceinline__ bool live() const { return t < count; }
    __device__ __forceinline__ void skip(int n)
    {
        for (k += n; live() && k >= x.kb;) {
            k -= x.kb;
            t += stride;
            if (t < count) x = tiles.at(t);
        }
    }
};

// Pair: one warp copies the scales of A, two those of B's rows 0 .. 127 and
// 128 .. 223 (both CTAs hold all of B's).  Otherwise one A, one B.  The fence
// that hands a stage to the tensor core waits for the warp's loads under way,
// so two sets of warps take the stages in turn: each has two stages' time.
template <int kMode, bool kPair>
__device__ __forceinline__ void copy_scales(const Tiles<kMode, kPair> &tiles, const Args &args, uint8_t *stages,
                                            uint64_t *full, uint64_t *empty, volatile int *abort_flag, int first,
                                            int stride, int count, uint32_t rank)
{
    using C = Cfg<kMode, kPair>;
    constexpr bool kAny = kMode == kForward4Any;
    constexpr int P = 2;  // a set's stages ahead
    constexpr int WORDS = (kPair ? 16 : 8) + (kAny ? 4 : 0);  // a lane's words of a stage
    const int part = ((threadIdx.x >> 5) - 8) % C::SCALE_WARPS, set = ((threadIdx.x >> 5) - 8) / C::SCALE_WARPS;
    const int lane = threadIdx.x & 31;
    const int J = kPair ? 2 : 128 / tiles.h;
    Walk<kMode, kPair> now(tiles, first, stride, count);
    now.skip(set);
    Walk<kMode, kPair> ahead = now;
    uint32_t w[P][WORDS];

    auto rows = [&](const Walk<kMode, kPair> &at) {
        ScaleRows s;
        s.stride = args.scale_bytes;
        s.byte0 = at.k * J * 8;
        if (part == 0) {
            const int c = at.x.c0 + static_cast<int>(rank) * 128 + lane;
            s.base = args.a_scales;
            s.total = static_cast<int64_t>(args.E) * args.cols * s.stride;
            s.row = static_cast<int64_t>(at.x.e) * args.cols + c;
            s.live = args.cols - c;
        } else {
            const int r = 128 * (part - 1) + lane;
            s.base = args.b_scales;
            s.total = static_cast<int64_t>(args.T) * s.stride;
            s.row = at.x.r0 + r;
            s.live = at.x.valid - r;
        }
        return s;
    };
    auto load = [&](uint32_t *v) {
        if (!ahead.live()) return;
        const ScaleRows s = rows(ahead);
        if (kPair) load_scales<kAny, 4, 4>(s, v);
        else if (J == 1 && part == 0) load_scales<kAny, 4, 2>(s, v);
        else if (J == 1) load_scales<kAny, 2, 2>(s, v);
        else if (J == 2 && part == 0) load_scales<kAny, 2, 4>(s, v);
        else if (J == 2) load_scales<kAny, 1, 4>(s, v);
        else load_scales<kAny, 1, 8>(s, v);
        ahead.skip(C::SCALE_SETS);
    };
#pragma unroll
    for (int p = 0; p < P; ++p) load(w[p]);
    bool ok = true;
    for (int g0 = set; ok && now.live(); g0 += P * C::SCALE_SETS) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            if (!ok || !now.live()) break;
            const int g = g0 + p * C::SCALE_SETS, slot = g % C::S;
            if (g >= C::S &&
                __any_sync(0xffffffffu, !mbar_wait(&empty[slot], ((g / C::S) - 1) & 1, args.timeout_ns, abort_flag))) {
                ok = false;
                break;
            }
            uint8_t *dst = stages + slot * C::STAGE + C::A_BYTES + C::B_BYTES + (part ? C::SA_BYTES : 0);
            const ScaleRows r = rows(now);
            if (kPair) store_scales<kAny, 4, 4>(part == 2 ? dst + 512 : dst, part ? 1024 : 512, lane, r, w[p]);
            else if (J == 1 && part == 0) store_scales<kAny, 4, 2>(dst, 512, lane, r, w[p]);
            else if (J == 1) store_scales<kAny, 2, 2>(dst, 512, lane, r, w[p]);
            else if (J == 2 && part == 0) store_scales<kAny, 2, 4>(dst, 512, lane, r, w[p]);
            else if (J == 2) store_scales<kAny, 1, 4>(dst, 512, lane, r, w[p]);
            else store_scales<kAny, 1, 8>(dst, 512, lane, r, w[p]);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (kPair) mbar_arrive_cluster(cluster_addr(&full[slot], 0));
                else mbar_arrive(&full[slot]);
            }
            now.skip(C::SCALE_SETS);
            load(w[p]);
        }
    }
    if (lane == 0 && !ok) {
        *abort_flag = 1;
        set_status(args.status, BSL_ERR_TIMEOUT);
    }
    __syncwarp();
}

template <int kMode, bool kPair>
__global__ void __launch_bounds__(Cfg<kMode, kPair>::THREADS, 1)
    k_grouped(const __grid_constant__ Maps maps, const Args args)
{
    using C = Cfg<kMode, kPair>;
    constexpr bool kAm = kMode == kInputGrad || kMode == kWeightGrad, kBm = kMode == kWeightGrad;  // M- / N-major operands
    extern __shared__ uint8_t smem_raw[];
    uint8_t *stages = align1024(smem_raw);
    uint8_t *outbuf = stages + C::S * C::STAGE;
    uint64_t *full = reinterpret_cast<uint64_t *>(outbuf + C::OUT);  // copies of a stage landed (leader)
    uint64_t *empty = full + C::S;                                   // MMAs of a stage finished (each CTA)
    uint64_t *afull = empty + C::S;                                  // accumulator complete (each CTA)
    uint64_t *aempty = afull + 2;                                    // accumulator read out (leader)
    uint64_t *drain = aempty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *h_slot = reinterpret_cast<int *>(tmem_slot + 2);
    int32_t *off = reinterpret_cast<int32_t *>(tmem_slot + 4);
    int32_t *start = off + kMaxExperts + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = kPair ? cluster_rank() : 0;
    const uint64_t tmo = args.timeout_ns;
    dependents_may_launch();

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::S; ++s) {
            mbar_init(&full[s], 1 + C::CG * C::SCALE_WARPS);
            mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&afull[a], 1);
            mbar_init(&aempty[a], 4 * C::CG);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_map(&maps.a[0]);
        tma_prefetch_map(&maps.b[8]);
        tma_prefetch_map(&maps.out);
    }
    if (warp == 1) {
        if (kPair) {
            tmem_alloc_pair(tmem_slot, C::TMEM);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(tmem_slot, C::TMEM);
            tmem_relinquish();
        }
    }
    wait_for_prior_grid();  // nothing above touched global memory
    if (warp == 0) {
        load_offsets(args.offsets, args.E, args.T, off, args.status);
        const int h = kPair ? 256 : pick_h(off, args.E, args.cols);
        const int nc = (args.cols + h - 1) / h, most = kPair ? C::BR : h / 2;
        tile_starts(args.E, start, [&](int e) {
            const int r = kMode == kWeightGrad ? args.rows : off[e + 1] - off[e];
            return (r + most - 1) / most * nc;
        });
        if (lane == 0) *h_slot = h;
    }
    tc_fence_before();
    __syncthreads();
    if (kPair) cluster_sync_all();  // the peer's barriers are initialised
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const Tiles<kMode, kPair> tiles = {off, start, args.E, *h_slot, args.cols, args.rows, args.depth};
    const int count = tiles.count();
    const int first = blockIdx.x / C::CG, stride = gridDim.x / C::CG;
    const int J = kPair ? 1 : 128 / tiles.h;  // 64-k blocks per stage

    if (warp == 0 || warp == 2) {
        // ------------------------------------------------------------ producers: warp 0 copies A, warp 2 B
        if (lane == 0) {
            const bool is_a = warp == 0;
            bool ok = true;
            int g = 0;  // stages issued
            int mapped = -1;
            // one strip a copy, two strips a copy
            const CUtensorMap *one = is_a ? &maps.a[kPair ? 1 : tiles.h == 128 ? 0 : tiles.h == 64 ? 1 : 2] : &maps.b[8];
            const CUtensorMap *two = &maps.a[0];
            for (int t = first; ok && t < count; t += stride) {
                const Tile x = tiles.at(t);
                if (kBm && x.kb > 0 && x.e != mapped) {
                    mapped = x.e;
                    one = args.expert_maps + 4 * static_cast<size_t>(x.e) + is_a;
                    two = one + 2;
                    asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(one) : "memory");
                    asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(two) : "memory");
                }
                const int half = x.n / C::CG;  // rows of B in this CTA
                const int at = is_a ? x.c0 + static_cast<int>(rank) * 128
                                    : x.r0 + static_cast<int>(rank) * half;
                if (kPair) {
                    const bool mn = is_a ? kAm : kBm;  // M- or N-major
                    const int plane = is_a && !kBm ? x.e : 0;
                    const int rows = is_a ? 128 : half;
                    const int strips = kBm && !is_a ? (half + 63) / 64 : 2;
                    const uint32_t bytes = 2 * (32768 + (kBm ? (half + 63) / 64 * 16384 : 256 * half));
                    // M-/N-major strips are whole along the features, K-major ones along k
                    const int wide = is_a ? args.cols : args.rows;
                    const bool aligned = mn && strips == 2 && at % 64 == 0 && (wide % 64 == 0 || at + 128 <= wide);
                    if (!is_a && !kBm) two = &maps.b[half / 16 - 1];  // exactly the tile's rows
                    for (int k = 0; k < x.kb; ++k, ++g) {
                        const int slot = g % C::S;
                        if (g >= C::S && !mbar_wait(&empty[slot], ((g / C::S) - 1) & 1, tmo, abort_flag)) {
                            ok = false;
                            break;
                        }
                        uint8_t *dst = stages + slot * C::STAGE + (is_a ? 0 : C::A_BYTES);
                        if (is_a && rank == 0) mbar_arrive_expect_tx(&full[slot], bytes);
                        const uint32_t bar = cluster_addr(&full[slot], 0);
                        if (mn) {
                            if (aligned)
                                tma_load_4d_pair(dst, two, bar, 0, k * 128, at / 64, plane);
                            else
                                for (int i = 0; i < strips; ++i)
                                    tma_load_3d_pair(dst + i * 16384, one, bar, at + 64 * i, k * 128, plane);
                        } else if (x.k % 64 == 0 || k * 128 + 128 <= x.k) {
                            tma_load_4d_pair(dst, two, bar, 0, at, k * 2, plane);
                        } else {  // the last stage of a k that ends inside a strip
                            for (int i = 0; i < 2; ++i)
                                for (int r = 0; r < rows; r += is_a ? 128 : C::BOX)
                                    tma_load_3d_pair(dst + (i * rows + r) * 128, one, bar, k * 128 + 64 * i, at + r, plane);
                        }
                    }
                } else {
                    const int boxes = (half + C::BOX - 1) / C::BOX;
                    const uint32_t bytes = C::A_BYTES + J * boxes * C::BOX * 128;
                    for (int k = 0; k < x.kb; ++k, ++g) {
                        const int slot = g % C::S;
                        if (g >= C::S && !mbar_wait(&empty[slot], ((g / C::S) - 1) & 1, tmo, abort_flag)) {
                            ok = false;
                            break;
                        }
                        uint8_t *sa = stages + slot * C::STAGE, *sb = sa + C::A_BYTES;
                        if (is_a) {
                            mbar_arrive_expect_tx(&full[slot], bytes);
                            for (int j = 0; j < J; ++j)
                                tma_load_3d(sa + j * tiles.h * 128, one, &full[slot], (k * J + j) * 64, at, x.e);
                        } else {
                            for (int j = 0; j < J; ++j)
                                for (int i = 0; i < boxes; ++i)
                                    tma_load_3d(sb + (j * boxes + i) * C::BOX * 128, one, &full[slot],
                                                (k * J + j) * 64, at + i * C::BOX, 0);
                        }
                    }
                }
            }
            if (!ok) {
                *abort_flag = 1;
                set_status(args.status, BSL_ERR_TIMEOUT);
            } else if (is_a) {  // the MMAs' arrivals on this CTA's barriers are in
                for (int s = 0; s < C::S && s < g; ++s) {
                    const int fills = (g - s + C::S - 1) / C::S;
                    if (!mbar_wait(&empty[s], (fills - 1) & 1, tmo, abort_flag))
                        set_status(args.status, BSL_ERR_TIMEOUT);
                }
            }
            // every copy lands before shared memory is released: the last fill of
            // each slot is the newest phase of its barrier, which the leader holds
            if (is_a && rank == 0)
                for (int s = 0; s < C::S && s < g; ++s) {
                    const int fills = (g - s + C::S - 1) / C::S;
                    if (!mbar_wait(&full[s], (fills - 1) & 1, tmo, nullptr)) set_status(args.status, BSL_ERR_TIMEOUT);
                }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if (rank == 0) {
            const uint32_t lead = lane == 0;
            bool ok = true;
            int g = 0, it = 0;
            for (int t = first; ok && t < count; t += stride) {
                const Tile x = tiles.at(t);
                if (x.kb == 0) continue;  // a sum over no rows: the epilogue writes zeros
                const int acc = it & 1;
                if (it >= 2 && __any_sync(0xffffffffu, !mbar_wait(&aempty[acc], ((it >> 1) - 1) & 1, tmo, abort_flag))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t idesc = C::F4 ? make_idesc_mx4(128 * C::CG, x.n) : make_idesc_bf16(128 * C::CG, x.n, kAm, kBm);
                const uint32_t d = tmem + acc * C::BR;
                for (int k = 0; k < x.kb; ++k, ++g) {
                    const int slot = g % C::S;
                    if (__any_sync(0xffffffffu, !mbar_wait(&full[slot], (g / C::S) & 1, tmo, abort_flag))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a0 = smem_u32(stages + slot * C::STAGE), b0 = a0 + C::A_BYTES;
                    // K-major: 8-row atoms 1024 bytes apart, a K step of 16 is 32 bytes along the row, a strip
                    // its rows x 128 bytes; M-major: strips 16384 bytes apart, a K step is 16 rows of 128 bytes
                    const uint64_t ad = make_sdesc(a0, kAm ? 16384 : 16, 1024, kLayoutSw128);
                    const uint64_t bd = make_sdesc(b0, kBm ? 16384 : 16, 1024, kLayoutSw128);
                    const uint32_t alo = static_cast<uint32_t>(ad), ahi = static_cast<uint32_t>(ad >> 32);
                    const uint32_t blo = static_cast<uint32_t>(bd), bhi = static_cast<uint32_t>(bd >> 32);
                    const uint32_t sa_t = tmem + C::SA_COL, sb_t = tmem + C::SB_COL;
                    if (C::F4) {  // the stage's scales to TMEM, in order with the MMAs around them
                        const uint64_t sc = make_sdesc(b0 + C::B_BYTES, 0, 128, 0);
                        const uint32_t lo = static_cast<uint32_t>(sc), hi = static_cast<uint32_t>(sc >> 32);
                        const int left = (x.k - k * 128 + 31) / 32;  // chunks of 128 elements
                        const int chunks = !kPair ? 2 * J : left < 4 ? left : 4;
                        for (int i = 0; i < chunks; ++i) {
                            scales_to_tmem<kPair>(lead, sa_t + 4 * i, lo + 32 * i, hi);
                            if (kPair) {
                                scales_to_tmem<kPair>(lead, sb_t + 8 * i, lo + C::SA_BYTES / 16 + 64 * i, hi);
                                if (x.n > 128) scales_to_tmem<kPair>(lead, sb_t + 8 * i + 4, lo + C::SA_BYTES / 16 + 64 * i + 32, hi);
                            } else {
                                scales_to_tmem<kPair>(lead, sb_t + 4 * i, lo + C::SA_BYTES / 16 + 32 * i, hi);
                            }
                        }
                    }
                    if (kPair) {
                        const uint32_t bs = x.n / 2 * 8;  // K-major B: a strip of half the rows, in 16-byte units
                        auto mma = [&](int i) {
                            if (C::F4)
                                umma_mx4<true>(lead, d, alo + (i >> 2) * 1024 + (i & 3) * 2, ahi,
                                               blo + (i >> 2) * bs + (i & 3) * 2, bhi, idesc | (i & 1) * kSecondScales,
                                               sa_t + (i >> 1) * 4, sb_t + (i >> 1) * 8, (k | i) != 0);
                            else
                                umma_bf16_lo_lead_pair(lead, d, alo + (kAm ? i * 128 : (i >> 2) * 1024 + (i & 3) * 2), ahi,
                                                       blo + (kBm ? i * 128 : (i >> 2) * bs + (i & 3) * 2), bhi, idesc,
                                                       (k | i) != 0);
                        };
                        const int left = x.k - k * 128;
                        if (left >= 128) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) mma(i);
                        } else {  // the copies filled the rest with zeros
                            for (int i = 0; 16 * i < left; ++i) mma(i);
                        }
                        umma_commit_lead_pair(lead, &empty[slot]);
                    } else {
                        const uint32_t aj = tiles.h * 8, bj = (x.n + C::BOX - 1) / C::BOX * C::BOX * 8;
                        for (int j = 0; j < J; ++j)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (C::F4)
                                    umma_mx4<false>(lead, d, alo + j * aj + i * 2, ahi, blo + j * bj + i * 2, bhi,
                                                    idesc | (i & 1) * kSecondScales, sa_t + (2 * j + (i >> 1)) * 4,
                                                    sb_t + (2 * j + (i >> 1)) * 4, (k | j | i) != 0);
                                else
                                    umma_bf16_lo_lead(lead, d, alo + j * aj + i * 2, ahi, blo + j * bj + i * 2, bhi, idesc,
                                                  (k | j | i) != 0);
                        umma_commit_lead(lead, &empty[slot]);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (kPair) umma_commit_lead_pair(lead, &afull[acc]);
                else umma_commit_lead(lead, &afull[acc]);
                __syncwarp();
                ++it;
            }
            if (lane == 0 && !ok) {
                *abort_flag = 1;
                set_status(args.status, BSL_ERR_TIMEOUT);
            }
            // every MMA is complete before TMEM and shared memory are released
            if (kPair) umma_commit_lead_pair(lead, drain);
            else umma_commit_lead(lead, drain);
            if (lane == 0 && !mbar_wait(drain, 0, tmo, nullptr)) set_status(args.status, BSL_ERR_TIMEOUT);
        }
        __syncwarp();
    } else if (warp == 3) {
        // ------------------------------------------------------------ rows of no expert
        if (kMode != kWeightGrad && args.zero_rest) {
            zero_range(args.out, 0, static_cast<int64_t>(off[0]) * args.cols, lane);
            zero_range(args.out, static_cast<int64_t>(off[args.E]) * args.cols,
                       static_cast<int64_t>(args.T) * args.cols, lane);
        }
        __syncwarp();
    } else if (C::F4 && warp >= 8) {
        if constexpr (C::F4) copy_scales<kMode, kPair>(tiles, args, stages, full, empty, abort_flag, first, stride, count, rank);
    } else {
        // ------------------------------------------------------------ epilogue
        // Warp q reads TMEM lanes 32q .. 32q+31: features c0 + 32q + lane of its CTA.
        const int q = warp & 3;
        uint8_t *wbuf = outbuf + q * 2 * C::CHUNK;
        const uint32_t lanes = static_cast<uint32_t>(32 * q) << 16;
        bool ok = true;
        int it = 0, ob = 0;
        for (int t = first; ok && t < count; t += stride) {
            const Tile x = tiles.at(t);
            const int c = x.c0 + static_cast<int>(rank) * 128 + 32 * q;
            const bool mine = c < args.cols && (kPair || 32 * q < tiles.h);
            const float bv = args.bias && mine && c + lane < args.cols
                                 ? __bfloat162float(args.bias[static_cast<int64_t>(x.e) * args.cols + c + lane]) : 0.f;
            const int acc = it & 1;
            if (x.kb > 0 && __any_sync(0xffffffffu, !mbar_wait(&afull[acc], (it >> 1) & 1, tmo, abort_flag))) {
                ok = false;
                break;
            }
            tc_fence_after();
            const int chunks = mine ? (x.valid + 31) / 32 : 0;
            for (int i = 0; i < chunks; ++i) {
                uint32_t v[32];
                if (x.kb > 0) {
                    tmem_ld32(tmem + lanes + acc * C::BR + i * 32, v);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int u = 0; u < 32; ++u) v[u] = 0;
                }
                if (lane == 0) bulk_wait_group_read<1>();  // the chunk's buffer was read out
                __syncwarp();
                uint8_t *dst = wbuf + ob * C::CHUNK;
                stage_chunk(dst, v, bv, lane);
                const int left = x.valid - 32 * i;
                if (kMode == kWeightGrad || left >= 32) {  // dW's map ends with the expert's rows
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        tma_store_3d(&maps.out, dst, c, x.r0 + 32 * i, kMode == kWeightGrad ? x.e : 0);
                } else {
                    __syncwarp();
                    store_rows(args.out + static_cast<int64_t>(x.r0 + 32 * i) * args.cols + c, args.cols, dst, left, args.cols - c, lane);
                }
                if (lane == 0) bulk_commit_group();  // one group a chunk, an empty one for plain stores
                ob ^= 1;
            }
            if (x.kb > 0) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (kPair) mbar_arrive_cluster(cluster_addr(&aempty[acc], 0));
                    else mbar_arrive(&aempty[acc]);
                }
                ++it;
            }
        }
        if (lane == 0) {
            if (!ok) {
                *abort_flag = 1;
                set_status(args.status, BSL_ERR_TIMEOUT);
            }
            bulk_wait_group<0>();
        }
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (kPair) {
        // the leader's last arrival on this CTA is in before the CTA may end
        if (rank != 0 && threadIdx.x == 0 && !mbar_wait(drain, 0, tmo, nullptr))
            set_status(args.status, BSL_ERR_TIMEOUT);
        __syncthreads();
        cluster_sync_all();  // no MMA, copy or arrival of the pair is left
    }
    if (warp == 1) {
        tc_fence_after();
        if (kPair) tmem_dealloc_pair(tmem, C::TMEM);
        else tmem_dealloc(tmem, C::TMEM);
    }
}

// ------------------------------------------------------------ host

inline bool map_rows(CUtensorMap *m, const void *p, int64_t cols, int64_t rows, uint32_t box_cols, uint32_t box_rows, int swizzle)
{
    return make_map_3d(m, p, cols, rows, 1, cols * 2, cols * 2 * rows, box_cols, box_rows, swizzle);
}

// Maps of a forward pass: the weight [E][N][depth], the rows [T][depth] and the output [T][N], two-byte columns.
inline bool forward_maps(Maps &m, const void *weight, int64_t N, int64_t depth, int64_t E, const void *X, int64_t T,
                         void *Y, bool pair)
{
    bool good = map_rows(&m.b[8], X, depth, T, 64, 16, 128) && map_rows(&m.out, Y, N, T, 32, 32, 0);
    if (pair) {
        good = good && make_strip_map(&m.a[0], weight, depth, N, E, 128, 2) &&
               make_map_3d(&m.a[1], weight, depth, N, E, depth * 2, depth * 2 * N, 64, 128, 128);
        for (int i = 0; i < 8; ++i) good = good && make_strip_map(&m.b[i], X, depth, T, 1, 16 * (i + 1), 2);
    } else {
        for (int i = 0; i < 3; ++i)
            good = good && make_map_3d(&m.a[i], weight, depth, N, E, depth * 2, depth * 2 * N, 64, 128 >> i, 128);
    }
    return good;
}

template <int kMode, bool kPair>
bsl_status run(const Maps &maps, const Args &args, cudaStream_t s)
{
    using C = Cfg<kMode, kPair>;
    auto kern = k_grouped<kMode, kPair>;
    const bsl_status sa = set_smem_once(reinterpret_cast<const void *>(kern), C::SMEM);
    if (sa != BSL_OK) return sa;
    const int grid = num_sms() / C::CG * C::CG;
    return cuda_status(kPair ? launch_dependent_cluster(kern, grid, 2, C::THREADS, C::SMEM, s, maps, args)
                             : launch_dependent(kern, grid, C::THREADS, C::SMEM, s, maps, args));
}

}  // namespace
}  // namespace bsl
