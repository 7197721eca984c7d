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
// The MMA's N may be any multiple of 32, so a tile with few rows costs few
// rows: an expert's rows are spread evenly over the fewest tiles of 256.  Rows of
// the next expert that a copy brings along only reach accumulator columns
// that are never stored.  For the weight gradient, whose ragged index is
// summed over, a row behind the expert's last one must be zero in both operands
// (a NaN there must not meet a zero), up to the next multiple of 16 rows, the k
// of an MMA.  So an expert's last stage, if it is not whole, comes in copies of
// 64, 32, .. 1 rows, as the rows left have ones in binary, and the zeros behind
// them in copies from behind the matrix.
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
// Clusters of two CTAs work on tiles of 256 features x up to 256 rows
// (cta_group::2, M = 256; each CTA holds its 128 rows of A and half of B) with
// a ring of stages of 128 k (three of full tiles).  With many rows the tensor pipe bounds it, as long as
// the copies keep up (32 KB per 64 k and SM, 64 bytes a clock), and those go
// by their number: an operand's stage is one copy of 32 KB, two strips of
// 128-byte rows.  At 16384 x 4096 x 14336, 8 experts, kernels back to back
// (clock held by power at 1.1-1.3 GHz): one 32 KB copy 1412 / 1459 / 1460 us
// for the three, copies of 16 KB and stages of 64 k 1460 / 1575 / 1540, of 8
// KB (gradients) 1775.  With few rows the weight's bytes bound it: 64 rows of
// 16 experts of 11008 x 4096 take 222 us (6.5 TB/s).  There, too, the pair is
// ahead of one CTA on tiles of 128 features (236 against 240 us with three
// stages; 93 against 110 us with 4-bit operands).
//
// Waiting costs: a waiting warp polls shared memory.  So one warp of a group
// waits and the others stand at a named barrier (4-bit, 8192 x 4096 x 14336:
// 236 against 240 us, and 293 with waits that spin).
//
// Every wait is bounded (BSL_ERR_TIMEOUT in the status word, then all roles
// leave through an abort flag, and the CTAs end when no copy can be under way).
#pragma once

#include "common.cuh"
#include "grouped.cuh"
#include "internal.h"

namespace bsl {
namespace {

// 4-bit operands by the units that a row of scales (K / 32 bytes) is whole in: kForward4 16 bytes (K a multiple of
// 512), kForward4By8, kForward4By4, kForward4Any any number
enum Mode { kForward, kInputGrad, kWeightGrad, kForward4, kForward4By8, kForward4By4, kForward4Any };

template <int kMode>
struct Cfg {
    static constexpr bool F4 = kMode >= kForward4;
    static constexpr bool AM = kMode == kInputGrad || kMode == kWeightGrad;  // A is M-major
    static constexpr bool BN = kMode == kWeightGrad;                         // B is N-major
    static constexpr int BC = 256;                   // features per tile
    static constexpr int BR = F4 ? 192 : 256;        // rows per tile, at most (4 bits: TMEM holds scales too)
    static constexpr int STEP = 32;                  // granularity of the rows (MMA N)
    static constexpr int BK = 128;                   // k per stage (two-byte columns)
    static constexpr int A_BYTES = 128 * BK * 2;
    static constexpr int B_BYTES = BR / 2 * BK * 2;
    static constexpr int RING = (F4 ? 180 : 192) * 1024;  // three stages of full tiles, up to S of smaller ones
    static constexpr int S = F4 ? 4 : 5;             // (4 bits: 5 are no faster, and 0.7 us slower for one row)
    // two accumulators, then a ring of scales: half a stage (256 elements of k), 8 columns of A's and 16 of B's
    static constexpr int SR = F4 ? 5 : 0, SC_COL = 2 * BR, SC_COLS = 24;
    static constexpr int TMEM = 512;
    static constexpr int CHUNK = 32 * 32 * 2;
    static constexpr int OUT = 4 * 2 * CHUNK;        // two chunks per epilogue warp
    static constexpr int SETS = 2;                   // of four warps that bring the scales of stages in turn
    static constexpr int RAW = F4 ? SETS * 2 * (128 + BR) * 16 : 0;  // two stages' scales a set, 16 bytes a row
    static constexpr int BARS = (2 * S + 2 * SR + 5) * 8 + 16;
    static constexpr int SMEM = 1024 + RING + OUT + RAW + BARS + 2 * (kMaxExperts + 1) * 4;
    static constexpr int THREADS = F4 ? 256 + SETS * 128 : 256;
    static_assert(SMEM <= 227 * 1024, "shared memory");
    static_assert(3 * (A_BYTES + B_BYTES) <= RING, "stages");
    static_assert(A_BYTES % 1024 == 0 && B_BYTES % 1024 == 0, "swizzle atoms");
    static_assert(SC_COL + SR * SC_COLS <= TMEM, "TMEM columns");
};

struct Maps {
    CUtensorMap a[2];   // A: two strips a copy, one strip (128 rows of K, or of features, each)
    CUtensorMap b[16];  // K-major B: b[i] two strips of 16 (i + 1) rows, b[8 + i] one, where k ends inside one
                        // N-major B: b[0], b[1] as a[0], a[1]; b[2 + j] one strip of 64 >> j rows, b[9 + j] of A
    CUtensorMap out;
};

struct Args {
    const int32_t *offsets;
    const __nv_bfloat16 *bias;
    __nv_bfloat16 *out;
    int32_t *status;
    int32_t T, E;
    int32_t cols, rows, depth;           // of the product; the ragged one is unused
    int32_t zero_rest;
    const uint8_t *a_scales, *b_scales;  // 4 bits: [E][cols][scale_bytes], [T][scale_bytes]
    int32_t scale_bytes;
    uint64_t timeout_ns;
};

struct Tile {
    int e, c0;     // expert, first feature
    int r0;        // first row: of the matrix, or of the expert's dW
    int n, valid;  // MMA N, rows that exist
    int k, kb;     // length of the sums, stages
    int k0;        // first k: the expert's first row in the weight gradient, else 0
};

// The tile list of a launch, the same in every CTA.
template <int kMode>
struct Tiles {
    const int32_t *off, *start;
    int E, cols, rows, depth;

    __device__ __forceinline__ Tile at(int t) const
    {
        using C = Cfg<kMode>;
        Tile x;
        x.e = expert_of(start, E, t);
        const int first = off[x.e], own = off[x.e + 1] - first;
        const int r = kMode == kWeightGrad ? rows : own;
        int ri, ci, r0;
        tile_place(t - start[x.e], (r + C::BR - 1) / C::BR, (cols + C::BC - 1) / C::BC, ri, ci);
        x.c0 = ci * C::BC;
        if (kMode == kWeightGrad) {  // whole strips: full tiles and a shorter last one
            r0 = ri * C::BR;
            x.n = r - r0 < C::BR ? (r - r0 + C::STEP - 1) / C::STEP * C::STEP : C::BR;
        } else {
            row_tile(r, C::BR, C::STEP, ri, r0, x.n);
        }
        x.valid = r - r0 < x.n ? r - r0 : x.n;
        x.r0 = kMode == kWeightGrad ? r0 : first + r0;
        x.k = kMode == kWeightGrad ? own : depth;
        x.kb = (x.k + C::BK - 1) / C::BK;
        x.k0 = kMode == kWeightGrad ? first : 0;
        return x;
    }
};

__device__ __forceinline__ uint8_t *align1024(uint8_t *p)
{
    return reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

// ------------------------------------------------------------ scales (4-bit forward)
//
// The block-scaled MMA takes its scales from TMEM: row r of 128 has, for 128
// elements of k (four blocks of 32), four bytes at lane r % 32, column r / 32,
// the same in all four quarters of the lanes.  The scales lie in plain rows in
// global memory, wherever an expert's rows begin.  Two sets of four warps, a
// warp per quarter of the lanes, bring the scales of stages there in turn: each
// warp loads a part of the rows (16 bytes of a row a lane and stage, some
// stages ahead), the four share them through shared memory, and each writes
// all of them to its lanes with tcgen05.st, half a stage at a time into a ring
// of five.
//
// Measured at 8192 x 4096 x 14336: copying them with tcgen05.cp (12 of 512
// bytes a stage, in order with the MMAs, some 55 clocks each) 260 us, this way
// 236, one set of warps 271; without any scales it would be 185.  An arrival
// with release semantics at the pair's barrier waits for the warp's loads
// under way: 529 us.
//
// Nothing is computed on what was loaded before its turn comes, so loads do
// not wait for one another.  Bytes past the row's end count as zeros (a scale
// of 2^-127 on zero codes; a NaN byte of the next row must not reach them),
// and so do rows that do not exist.

// W words of a row from byte0 on, of rows in whole units of V words.
template <int W, int V>
__device__ __forceinline__ void load_words(const uint8_t *base, int32_t stride, int64_t row, bool exists, int32_t byte0,
                                           uint32_t *w)
{
    const uint8_t *at = base + row * stride + byte0;
#pragma unroll
    for (int i = 0; i < W; i += V) {
        const bool in = exists && byte0 + 4 * i < stride;
        if constexpr (V == 4) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (in) v = load_global(reinterpret_cast<const uint4 *>(at + 4 * i));
            w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
        } else if constexpr (V == 2) {
            uint2 v = make_uint2(0, 0);
            if (in) v = load_global(reinterpret_cast<const uint2 *>(at + 4 * i));
            w[i] = v.x, w[i + 1] = v.y;
        } else {
            w[i] = 0;
            if (in) w[i] = load_global(reinterpret_cast<const uint32_t *>(at + 4 * i));
        }
    }
}

// Rows that start at any byte: the W + 1 aligned words around them, as far as
// they hold bytes of the row.  The last bytes of the array may fill no whole
// word and are read one by one.
template <int W>
__device__ __forceinline__ void load_words_any(const uint8_t *base, int64_t total, int32_t stride, int64_t row, bool exists,
                                               int32_t byte0, uint32_t *w)
{
    const int64_t at = row * stride + byte0;
    const int32_t skip = static_cast<int32_t>(at & 3), left = exists ? stride - byte0 + skip : 0;
    const uint8_t *p = base + (at - skip);
    const bool end = exists && total - at < 4 * W + 4;
    const int32_t whole = end ? static_cast<int32_t>(total - at) + skip : 4 * W + 4;
#pragma unroll
    for (int i = 0; i <= W; ++i) {
        w[i] = 0;
        if (4 * i < left && 4 * i + 4 <= whole) w[i] = load_global(reinterpret_cast<const uint32_t *>(p + 4 * i));
    }
    if (end) {
#pragma unroll
        for (int i = 0; i <= W; ++i)
            if (4 * i + 4 > whole)
                for (int b = 4 * i; b < whole && b < 4 * i + 4; ++b) w[i] |= static_cast<uint32_t>(p[b]) << (8 * (b & 3));
    }
}

// ... and, when they are stored, shifted into place and cut at the row's end.
template <int W>
__device__ __forceinline__ void shift_words(int32_t stride, int64_t row, int32_t byte0, const uint32_t *r, uint32_t *w)
{
    const uint32_t shift = (static_cast<uint32_t>(row) * static_cast<uint32_t>(stride) + static_cast<uint32_t>(byte0)) % 4 * 8;
    const int32_t left = stride - byte0;
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = __funnelshift_r(r[i], r[i + 1], shift);
    if (left < 4 * W) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const int32_t bytes = left - 4 * i;
            if (bytes < 4) w[i] &= bytes <= 0 ? 0 : (1u << (8 * bytes)) - 1u;
        }
    }
}

// Halves of a stage that hold elements.
__device__ __forceinline__ int halves(const Tile &x, int k) { return x.k - k * 128 > 64 ? 2 : 1; }

// A walk over this CTA's stages, tile after tile.
template <int kMode>
struct Walk {
    const Tiles<kMode> &tiles;
    int t, stride, count, k;
    Tile x;

    __device__ __forceinline__ Walk(const Tiles<kMode> &l, int first, int step, int n)
        : tiles(l), t(first), stride(step), count(n), k(0)
    {
        if (live()) x = tiles.at(t);
    }
    __device__ __forceinline__ bool live() const { return t < count; }
    __device__ __forceinline__ void next()
    {
        if (!live() || ++k < x.kb) return;
        k = 0;
        t += stride;
        if (live()) x = tiles.at(t);
    }
};

template <int kMode>
__device__ __forceinline__ void copy_scales(const Tiles<kMode> &tiles, const Args &args, uint8_t *raw, uint64_t *sfull,
                                            uint64_t *sempty, volatile int *abort_flag, int first, int stride, int count,
                                            uint32_t rank, uint32_t tmem)
{
    using C = Cfg<kMode>;
    constexpr bool kAny = kMode == kForward4Any;
    constexpr int V = kMode == kForward4 ? 4 : kMode == kForward4By8 ? 2 : 1;
    constexpr int W = 4, R = W + kAny;  // a row's words of a stage, and as loaded
    constexpr int P = 2;                // stages of its own that a set loads ahead
    constexpr int G = C::BR / 32;       // groups of 32 rows of B
    const int q = threadIdx.x / 32 & 3, set = threadIdx.x / 128 - 2, lane = threadIdx.x & 31;
    const int32_t bytes = args.scale_bytes;
    const int64_t a_total = static_cast<int64_t>(args.E) * args.cols * bytes, b_total = static_cast<int64_t>(args.T) * bytes;
    Walk<kMode> now(tiles, first, stride, count);
    int h = 0;  // halves of stages so far, the other set's too
    if (set && now.live()) {
        h = halves(now.x, now.k);
        now.next();
    }
    Walk<kMode> ahead = now;
    uint32_t w[P][3][R];

    // This warp's rows: 32q + lane of A, of B, and 128 + 32q + lane of B.
    struct Row {
        const uint8_t *base;
        int64_t total, row;
        bool exists;
    };
    auto rows = [&](const Walk<kMode> &at, int i) {
        Row r;
        if (i == 0) {
            const int c = at.x.c0 + static_cast<int>(rank) * 128 + 32 * q + lane;
            r.base = args.a_scales;
            r.total = a_total;
            r.row = static_cast<int64_t>(at.x.e) * args.cols + c;
            r.exists = c < args.cols;
        } else {
            const int b = 128 * (i - 1) + 32 * q + lane;
            r.base = args.b_scales;
            r.total = b_total;
            r.row = at.x.r0 + b;
            r.exists = b < at.x.valid;
        }
        return r;
    };
    auto load = [&](uint32_t(&v)[3][R]) {
        if (!ahead.live()) return;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const Row r = rows(ahead, i);
            if constexpr (kAny) load_words_any<W>(r.base, r.total, bytes, r.row, r.exists, 16 * ahead.k, v[i]);
            else load_words<W, V>(r.base, bytes, r.row, r.exists, 16 * ahead.k, v[i]);
        }
        ahead.next();
        ahead.next();
    };
#pragma unroll
    for (int p = 0; p < P; ++p) load(w[p]);
    bool ok = true;
    while (now.live()) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            if (!now.live()) break;
            uint4 *buf = reinterpret_cast<uint4 *>(raw) + (2 * set + p) * (128 + C::BR);
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                const int at = 32 * q + lane + 128 * i;
                if (at >= 128 + C::BR) break;
                if constexpr (kAny) {
                    const Row r = rows(now, i);
                    uint32_t v[W];
                    shift_words<W>(bytes, r.row, 16 * now.k, w[p][i], v);
                    buf[at] = make_uint4(v[0], v[1], v[2], v[3]);
                } else {
                    buf[at] = make_uint4(w[p][i][0], w[p][i][1], w[p][i][2], w[p][i][3]);
                }
            }
            // One warp waits for the stage's place in the ring (a waiting warp polls
            // shared memory, which the MMAs and copies need), the barrier lets the
            // others know.  All four reach every barrier, an aborted run's too;
            // behind the next one, this buffer has been read.  An mbarrier tells
            // neighbouring phases apart and no more: the set's last wait was for
            // half h - 3 - SR or a later one, and half h cannot be finished without it.
            const int n = halves(now.x, now.k);
            if (q == 0) {
                for (int i = 0; ok && i < n; ++i)
                    if (h + i >= C::SR && __any_sync(0xffffffffu, !mbar_wait(&sempty[(h + i) % C::SR], ((h + i) / C::SR - 1) & 1,
                                                                             args.timeout_ns, abort_flag)))
                        ok = false;
                if (lane == 0 && !ok) *abort_flag = 1;
                __syncwarp();
            }
            named_bar_sync(1 + set, 128);
            if (*abort_flag) ok = false;
            uint32_t a[4][4], b[8][4];  // [rows lane + 32 i][chunk of 128 elements]
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 v = buf[32 * i + lane];
                a[i][0] = v.x, a[i][1] = v.y, a[i][2] = v.z, a[i][3] = v.w;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint4 v = i < G && 32 * i < now.x.n ? buf[128 + 32 * i + lane] : make_uint4(0, 0, 0, 0);
                b[i][0] = v.x, b[i][1] = v.y, b[i][2] = v.z, b[i][3] = v.w;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (i >= n) break;
                const int slot = h % C::SR;
                if (ok) {
                    tc_fence_after();
                    uint32_t va[8], vb[16];
#pragma unroll
                    for (int c = 0; c < 4; ++c) va[c] = a[c][2 * i], va[4 + c] = a[c][2 * i + 1];
#pragma unroll
                    for (int c = 0; c < 8; ++c) vb[c] = b[c][2 * i], vb[8 + c] = b[c][2 * i + 1];
                    const uint32_t at = tmem + (static_cast<uint32_t>(32 * q) << 16) + C::SC_COL + slot * C::SC_COLS;
                    tmem_st8(at, va);
                    tmem_st16(at + 8, vb);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(cluster_addr(&sfull[slot], 0));
                }
                ++h;
            }
            now.next();
            if (now.live()) h += halves(now.x, now.k);
            now.next();
            load(w[p]);
        }
    }
    // the MMAs' last arrivals on this CTA's barriers are in before it may end
    for (int s = 0; ok && s < C::SR && s < h; ++s)
        if (__any_sync(0xffffffffu, !mbar_wait(&sempty[s], ((h - s + C::SR - 1) / C::SR - 1) & 1, args.timeout_ns, abort_flag)))
            ok = false;
    if (lane == 0 && !ok) {
        *abort_flag = 1;
        set_status(args.status, BSL_ERR_TIMEOUT);
    }
    __syncwarp();
}

// Bytes of a stage in the ring, by the calling warp: the rows of B are those of
// the launch's largest tile.  What few rows leave free holds more stages: 64
// rows of 16 experts of 11008 x 4096 take 222 us with five, 236 with three.
template <int kMode>
__device__ __forceinline__ int stage_bytes(const int32_t *off, int32_t E)
{
    using C = Cfg<kMode>;
    if (kMode == kWeightGrad) return C::A_BYTES + C::B_BYTES;
    int top = 1;
    for (int e = threadIdx.x & 31; e < E; e += 32) top = max(top, off[e + 1] - off[e]);
    top = __reduce_max_sync(0xffffffffu, top);
    const int rows = top > C::BR ? C::BR : (top + C::STEP - 1) / C::STEP * C::STEP;
    return C::A_BYTES + rows / 2 * C::BK * 2;
}

// A place in the ring: slot, and the parity of the phase that fills it.
struct Place {
    int slot = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next(int S)
    {
        if (++slot == S) {
            slot = 0;
            parity ^= 1;
        }
    }
};

template <int kMode>
__global__ void __launch_bounds__(Cfg<kMode>::THREADS, 1)
    k_grouped(const __grid_constant__ Maps maps, const Args args)
{
    using C = Cfg<kMode>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *stages = align1024(smem_raw);
    uint8_t *outbuf = stages + C::RING;
    uint8_t *raw = outbuf + C::OUT;
    uint64_t *full = reinterpret_cast<uint64_t *>(raw + C::RAW);     // copies of a stage landed (leader)
    uint64_t *empty = full + C::S;                                   // MMAs of a stage finished (each CTA)
    uint64_t *afull = empty + C::S;                                  // accumulator complete (each CTA)
    uint64_t *aempty = afull + 2;                                    // accumulator read out (leader)
    uint64_t *sfull = aempty + 2;                                    // half a stage's scales in TMEM (leader)
    uint64_t *sempty = sfull + C::SR;                                // ... used (each CTA)
    uint64_t *drain = sempty + C::SR;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *ring_slot = reinterpret_cast<int *>(tmem_slot + 2);
    int32_t *off = reinterpret_cast<int32_t *>(tmem_slot + 4);
    int32_t *start = off + kMaxExperts + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const uint64_t tmo = args.timeout_ns;
    dependents_may_launch();

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < C::SR; ++s) {
            mbar_init(&sfull[s], 8);
            mbar_init(&sempty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&afull[a], 1);
            mbar_init(&aempty[a], 8);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_map(&maps.a[0]);
        tma_prefetch_map(&maps.out);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, C::TMEM);
        tmem_relinquish_pair();
    }
    wait_for_prior_grid();  // nothing above touched global memory
    fetch_offsets(args.offsets, args.E, args.T, off);
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        clamp_offsets(args.E, args.T, off, args.status);
        const int nc = (args.cols + C::BC - 1) / C::BC;
        tile_starts(args.E, start, [&](int e) {
            const int r = kMode == kWeightGrad ? args.rows : off[e + 1] - off[e];
            return (r + C::BR - 1) / C::BR * nc;
        });
        const int bytes = stage_bytes<kMode>(off, args.E);
        if (lane == 0) *ring_slot = bytes;
    }
    __syncthreads();
    cluster_sync_all();  // the peer's barriers are initialised
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const Tiles<kMode> tiles = {off, start, args.E, args.cols, args.rows, args.depth};
    const int count = start[args.E];
    const int first = blockIdx.x / 2, stride = gridDim.x / 2;
    const int stage = *ring_slot, S = C::RING / stage < C::S ? C::RING / stage : C::S;  // a stage's bytes, stages

    if (warp == 0 || warp == 2) {
        // ------------------------------------------------------------ producers: warp 0 copies A, warp 2 B
        if (lane == 0) {
            const bool is_a = warp == 0;
            const bool mn = is_a ? C::AM : C::BN;  // M- or N-major
            bool ok = true;
            int g = 0;  // stages issued
            Place at_ring;
            // one, two strips a copy
            const CUtensorMap *one = C::BN && !is_a ? &maps.b[1] : &maps.a[1], *two = C::BN && !is_a ? &maps.b[0] : &maps.a[0];
            Tile x, next;
            if (first < count) next = tiles.at(first);
            for (int t = first; ok && t < count; t += stride) {
                x = next;
                if (t + stride < count) next = tiles.at(t + stride);
                const int half = x.n / 2;  // rows of B in this CTA
                const int at = is_a ? x.c0 + static_cast<int>(rank) * 128 : x.r0 + static_cast<int>(rank) * half;
                const int plane = is_a && kMode != kWeightGrad ? x.e : 0;
                const int rows = is_a ? 128 : half;
                const int strips = C::BN && !is_a ? (half + 63) / 64 : 2;
                const uint32_t bytes = 2 * (C::A_BYTES + (C::BN ? (half + 63) / 64 * 16384 : 256 * half));
                // M- and N-major strips are whole along the features, K-major ones along k
                const int wide = is_a ? args.cols : args.rows;
                const bool aligned = mn && strips == 2 && at % 64 == 0 && (wide % 64 == 0 || at + 128 <= wide);
                if (!is_a && !C::BN) {  // exactly the tile's rows
                    two = &maps.b[half / 16 - 1];
                    one = two + 8;
                }
                for (int k = 0; k < x.kb; ++k, ++g, at_ring.next(S)) {
                    const int slot = at_ring.slot;
                    if (g >= S && !mbar_wait(&empty[slot], at_ring.parity ^ 1, tmo, abort_flag)) {
                        ok = false;
                        break;
                    }
                    uint8_t *dst = stages + slot * stage + (is_a ? 0 : C::A_BYTES);
                    const int left = x.k - k * 128, row = x.k0 + k * 128;
                    const bool rest = kMode == kWeightGrad && left < 128;  // of the expert's rows, not a whole stage
                    const int lines = (left + 15) / 16 * 16;               // ... and the zeros behind them
                    if (is_a && rank == 0) mbar_arrive_expect_tx(&full[slot], rest ? bytes / 128 * lines : bytes);
                    const uint32_t bar = cluster_addr(&full[slot], 0);
                    if (rest) {  // (the swizzle goes by the address, so a copy may begin at any line)
                        const CUtensorMap *part = &maps.b[is_a ? 9 : 2];
                        for (int i = 0; i < strips; ++i) {
                            uint8_t *to = dst + i * 16384;
                            int y = row;
                            for (int j = 0; j < 7; ++j)
                                if (left >> (6 - j) & 1) {
                                    tma_load_3d_pair(to, part + j, bar, at + 64 * i, y, 0);
                                    y += 64 >> j;
                                    to += 8192 >> j;
                                }
                            for (int j = 3; j < 7; ++j)
                                if ((lines - left) >> (6 - j) & 1) {
                                    tma_load_3d_pair(to, part + j, bar, at + 64 * i, args.T, 0);  // no such row: zeros
                                    to += 8192 >> j;
                                }
                        }
                    } else if (mn) {
                        if (aligned)
                            tma_load_4d_pair(dst, two, bar, 0, row, at / 64, plane);
                        else
                            for (int i = 0; i < strips; ++i)
                                tma_load_3d_pair(dst + i * 16384, one, bar, at + 64 * i, row, plane);
                    } else if (x.k % 64 == 0 || k * 128 + 128 <= x.k) {
                        tma_load_4d_pair(dst, two, bar, 0, at, k * 2, plane);
                    } else {  // the last stage of a k that ends inside a strip
                        for (int i = 0; i < 2; ++i)
                            tma_load_3d_pair(dst + i * rows * 128, one, bar, k * 128 + 64 * i, at, plane);
                    }
                }
            }
            if (!ok) {
                *abort_flag = 1;
                set_status(args.status, BSL_ERR_TIMEOUT);
            } else if (is_a) {  // the MMAs' arrivals on this CTA's barriers are in
                for (int s = 0; s < S && s < g; ++s) {
                    const int fills = (g - s + S - 1) / S;
                    if (!mbar_wait(&empty[s], (fills - 1) & 1, tmo, abort_flag))
                        set_status(args.status, BSL_ERR_TIMEOUT);
                }
            }
            // every copy lands before shared memory is released: the last fill of
            // each slot is the newest phase of its barrier, which the leader holds
            if (is_a && rank == 0)
                for (int s = 0; s < S && s < g; ++s) {
                    const int fills = (g - s + S - 1) / S;
                    if (!mbar_wait(&full[s], (fills - 1) & 1, tmo, nullptr)) set_status(args.status, BSL_ERR_TIMEOUT);
                }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (the leader's)
        if (rank == 0) {
            const uint32_t lead = lane == 0;
            // What the loops and the MMAs' operands depend on is the same in all lanes;
            // said so, they stay in uniform registers and an MMA is a few instructions
            const uint32_t tm = uniform(tmem);
            const int tiles_end = uniform(count), ring = uniform(S);
            const uint32_t bytes = uniform(static_cast<uint32_t>(stage));
            bool ok = true;
            Place at;
            int h = 0, it = 0;
            for (int t = first; ok && t < tiles_end; t += stride) {
                Tile x = tiles.at(t);
                x.n = uniform(x.n);
                x.k = uniform(x.k);
                x.kb = uniform(x.kb);
                if (x.kb == 0) continue;  // a sum over no rows: the epilogue writes zeros
                const int acc = it & 1;
                if (it >= 2 && __any_sync(0xffffffffu, !mbar_wait(&aempty[acc], ((it >> 1) - 1) & 1, tmo, abort_flag))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t idesc = C::F4 ? make_idesc_mx4(256, x.n) : make_idesc_bf16(256, x.n, C::AM, C::BN);
                const uint32_t d = tm + acc * C::BR;
                const uint32_t bs = x.n / 2 * 8;  // K-major B: a strip of half the rows, in 16-byte units
                for (int k = 0; k < x.kb; ++k, at.next(ring)) {
                    const int slot = at.slot;
                    if (__any_sync(0xffffffffu, !mbar_wait(&full[slot], at.parity, tmo, abort_flag))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a0 = smem_u32(stages) + slot * bytes, b0 = a0 + C::A_BYTES;
                    // K-major: 8-row atoms 1024 bytes apart, a K step of 32 bytes along the row, a strip its
                    // rows x 128 bytes; M- and N-major: strips 16384 bytes apart, a K step of 16 rows of 128 bytes
                    const uint64_t ad = make_sdesc(a0, C::AM ? 16384 : 16, 1024, kLayoutSw128);
                    const uint64_t bd = make_sdesc(b0, C::BN ? 16384 : 16, 1024, kLayoutSw128);
                    const uint32_t alo = static_cast<uint32_t>(ad), ahi = static_cast<uint32_t>(ad >> 32);
                    const uint32_t blo = static_cast<uint32_t>(bd), bhi = static_cast<uint32_t>(bd >> 32);
                    auto mma = [&](int i, uint32_t sc) {
                        const uint32_t al = alo + (C::AM ? i * 128 : (i >> 2) * 1024 + (i & 3) * 2);
                        const uint32_t bl = blo + (C::BN ? i * 128 : (i >> 2) * bs + (i & 3) * 2);
                        if (C::F4)
                            umma_mx4_lead_pair(lead, d, al, ahi, bl, bhi, idesc | (i & 1) * kSecondScales,
                                               sc + (i >> 1 & 1) * 4, sc + 8 + (i >> 1 & 1) * 8, (k | i) != 0);
                        else
                            umma_bf16_lo_lead_pair(lead, d, al, ahi, bl, bhi, idesc, (k | i) != 0);
                    };
                    const int left = x.k - k * 128;  // the copies filled the rest of the stage with zeros
                    if constexpr (C::F4) {
                        // halves are handed over in order: the last one's barrier tells for both
                        const int n = halves(x, k), s0 = h % C::SR, s1 = (h + 1) % C::SR, last = h + n - 1;
                        if (__any_sync(0xffffffffu, !mbar_wait(&sfull[last % C::SR], (last / C::SR) & 1, tmo, abort_flag))) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
#pragma unroll
                        for (int i = 0; i < 4; ++i) mma(i, tm + C::SC_COL + s0 * C::SC_COLS);
                        umma_commit_lead_pair(lead, &sempty[s0]);
                        if (n == 2) {
#pragma unroll
                            for (int i = 4; i < 8; ++i) mma(i, tm + C::SC_COL + s1 * C::SC_COLS);
                            umma_commit_lead_pair(lead, &sempty[s1]);
                        }
                        h += n;
                    } else if (left >= 128) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) mma(i, 0);
                    } else {
                        for (int i = 0; 16 * i < left; ++i) mma(i, 0);
                    }
                    umma_commit_lead_pair(lead, &empty[slot]);
                    __syncwarp();
                }
                if (!ok) break;
                umma_commit_lead_pair(lead, &afull[acc]);
                __syncwarp();
                ++it;
            }
            if (lane == 0 && !ok) {
                *abort_flag = 1;
                set_status(args.status, BSL_ERR_TIMEOUT);
            }
            // every MMA is complete before TMEM and shared memory are released
            umma_commit_lead_pair(lead, drain);
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
        if constexpr (C::F4) copy_scales<kMode>(tiles, args, raw, sfull, sempty, abort_flag, first, stride, count, rank, tmem);
    } else {
        // ------------------------------------------------------------ epilogue
        // Warp q reads TMEM lanes 32q .. 32q+31: features c0 + 32q + lane of its CTA.
        const int q = warp & 3;
        uint8_t *wbuf = outbuf + q * 2 * C::CHUNK;
        const uint32_t lanes = static_cast<uint32_t>(32 * q) << 16;
        bool ok = true;
        int it = 0, ob = 0;
        for (int t = first; t < count; t += stride) {
            const Tile x = tiles.at(t);
            const int c = x.c0 + static_cast<int>(rank) * 128 + 32 * q;
            const float bv = args.bias && c + lane < args.cols
                                 ? __bfloat162float(args.bias[static_cast<int64_t>(x.e) * args.cols + c + lane]) : 0.f;
            const int acc = it & 1;
            if (x.kb > 0) {
                // one warp waits (a waiting warp polls shared memory, which the MMAs and
                // copies need); all four come to every tile's barrier, an aborted run's too
                // (a whole tile's sum: its limit grows by 4 us a stage, which takes one at most)
                const uint64_t limit = tmo + 4096ull * static_cast<uint32_t>(x.kb);
                if (ok && q == 0 && __any_sync(0xffffffffu, !mbar_wait(&afull[acc], (it >> 1) & 1, limit, abort_flag)) &&
                    lane == 0)
                    *abort_flag = 1;
                __syncwarp();
                named_bar_sync(3, 128);
                ++it;
            }
            if (*abort_flag) ok = false;
            if (!ok) continue;
            tc_fence_after();
            const int chunks = c < args.cols ? (x.valid + 31) / 32 : 0;
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
                if (kMode == kWeightGrad || left >= 32) {  // dW's map ends with each plane's rows
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        tma_store_3d(&maps.out, dst, c, x.r0 + 32 * i, kMode == kWeightGrad ? x.e : 0);
                } else {
                    __syncwarp();
                    store_rows(args.out + static_cast<int64_t>(x.r0 + 32 * i) * args.cols + c, args.cols, dst, left,
                               args.cols - c, lane);
                }
                if (lane == 0) bulk_commit_group();  // one group a chunk, an empty one for plain stores
                ob ^= 1;
            }
            if (x.kb > 0) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(cluster_addr(&aempty[acc], 0));
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
    // the leader's last arrival on this CTA is in before the CTA may end
    if (rank != 0 && threadIdx.x == 0 && !mbar_wait(drain, 0, tmo, nullptr)) set_status(args.status, BSL_ERR_TIMEOUT);
    __syncthreads();
    // An aborted run's producers gave up one by one, and one of the four may have
    // started a copy of a stage that the leader never armed: no barrier tells of it
    // (a stage that is not armed is never multiplied, so both CTAs give up).
    // Such a copy ends by itself in some microseconds: wait a thousand.
    if (*abort_flag) {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000) __nanosleep(1000);
        __syncwarp();
    }
    cluster_sync_all();  // no MMA, copy or arrival of the pair is left
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, C::TMEM);
    }
}

// ------------------------------------------------------------ host

// Rows [rows][cols] of two-byte columns, boxes of box_cols x box_rows.
inline bool map_rows(CUtensorMap *m, const void *p, int64_t cols, int64_t rows, uint32_t box_cols, uint32_t box_rows,
                     int swizzle)
{
    return make_map_3d(m, p, cols, rows, 1, cols * 2, cols * 2 * rows, box_cols, box_rows, swizzle);
}

// Maps of a pass over rows: the weight [E][N][K], the rows [T][depth] and the output [T][cols], two-byte columns.
inline bool row_maps(Maps &m, const void *weight, int64_t E, int64_t N, int64_t K, const void *A, int64_t T, int64_t depth,
                     void *out, int64_t cols)
{
    bool good = make_strip_map(&m.a[0], weight, K, N, E, 128, 2) &&
                make_map_3d(&m.a[1], weight, K, N, E, K * 2, K * 2 * N, 64, 128, 128) &&
                map_rows(&m.out, out, cols, T, 32, 32, 0);
    // (a tile has no more than T rows, rounded up to 32)
    for (int i = 0; i < 8 && 32 * i < T; ++i)
        good = good && make_strip_map(&m.b[i], A, depth, T, 1, 16 * (i + 1), 2) &&
               (depth % 64 == 0 || map_rows(&m.b[8 + i], A, depth, T, 64, 16 * (i + 1), 128));
    return good;
}

template <int kMode>
bsl_status run(const Maps &maps, const Args &args, cudaStream_t s)
{
    using C = Cfg<kMode>;
    auto kern = k_grouped<kMode>;
    const bsl_status sa = set_smem_once(reinterpret_cast<const void *>(kern), C::SMEM);
    if (sa != BSL_OK) return sa;
    const int grid = num_sms() / 2 * 2;
    return cuda_status(launch_dependent_cluster(kern, grid, 2, C::THREADS, C::SMEM, s, maps, args));
}

}  // namespace
}  // namespace bsl
