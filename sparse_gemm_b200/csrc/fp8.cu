// fp8.cu -- products of 8-bit (e4m3) matrices with a scale for each block of 128
// (fp8_quant.cu gives the format), dense or grouped by expert:
//     forward          Y[t][n]  = sum_b sx[t][b] sw[n/128][b] sum_{k in b} x[t][k] w[n][k] (+ bias)
//     input gradient   dX[t][k] = sum_b sg[t][b] sw[b][k/128] sum_{n in b} g[t][n] w[n][k]
//
// The scales are fp32 numbers, which the tensor cores do not take, and change
// every 128 elements of the sum.  So each block's sum is an accumulator of its
// own in TMEM; sixteen warps bring it to registers, multiply it by the two
// scales and add it to the output's sum there, 32 bits throughout, while the
// MMAs fill the other accumulator.  The rows t go to the MMA's M side, the
// TMEM lanes: a block's scales, of the row and of the weight's tile, are then one
// number for all of a thread's columns.  (With the features on the lanes, as in the
// bf16 kernel, every column would need one of its own from shared memory.)
//
// Clusters of two CTAs work on tiles of up to 256 rows x 256 columns
// (cta_group::2, M = 256): each CTA holds half of the tile's rows, its 128 lanes,
// and half of the weight's columns.  A stage is one block, 16 KB of each
// operand.  An expert's rows are spread evenly over the fewest tiles, and copies
// bring exactly a tile's rows.  The weight is K-major in the forward and N-major
// in the gradient, the same codes for both.
//
// Persistent kernels, programmatic dependents, 20 warps a CTA:
//   warp 0      TMA producer (a ring of stages);
//   warp 1      MMA issuer and TMEM owner;
//   warp 2      the one that waits for the MMAs of a stage: the sums stand at a
//               named barrier (a waiting warp polls shared memory, which the MMAs and
//               copies need);
//   warp 3      products of the two scales of each row and block, some stages
//               ahead, into shared memory; then zeros for the rows of no expert, on
//               request;
//   warps 4-19  sums: warp 4 + 4 p + q owns lanes 32 q .. of columns 64 p ..
// Tiles are dealt round robin; no workspace is shared by calls, and every output
// is one sum in a fixed order.
//
// What bounds it with many rows is the turn of an accumulator, two of which fill
// TMEM: a stage takes 905 clocks (issue to issue, by clock() in a copy of this kernel), half a
// turn, and a tile's end 3260 more, while the sums write it, so 1010 a stage of 32-stage
// tiles.  With clocks at three points, which slow it to 1110 a stage, a turn is 1310 from the issue until
// the sums see the block, 680 until they have read it out (their FMAs take 280 of it) and 235
// until the next issue.  Measured at 8192 x 4096 x 14336: 502 us for single calls (1920 TFLOP/s), 566 in a
// row of them at 1556 MHz, which power holds back, 595 with the rows' conversion (17); MMAs and copies
// alone 305.  Steps and what they took: output by plain stores, which all SMs issue at
// the same time, 562, by copies from shared memory 545; without a split of the
// registers by setmaxnreg 502.  Eight sum warps with twice the columns took 530, and
// 800 to 1050 where the compiler spilled some of their 128 sums; MMAs of 128 columns
// with twice the accumulators 402 without any sums.  One waiting warp instead of
// sixteen is worth 380 against 428 with the sums left out, nothing with them (562, 561).
//
// Every wait is bounded (BSL_ERR_TIMEOUT in the status word, then all roles
// leave through an abort flag, and the CTAs end when no copy can be under way).
#include "common.cuh"
#include "grouped.cuh"
#include "internal.h"
#include "pair.cuh"

namespace bsl {
namespace {

constexpr int kBC = 256, kBR = 256;             // columns and rows of a tile
constexpr int kStep = 32;                       // granularity of the rows
constexpr int kBlock = 128;                     // elements that share a scale: a stage
constexpr int kWBytes = 128 * kBlock;           // a CTA's half of the weight's part of a stage
constexpr int kRing = 144 * 1024;
constexpr int kStages = 8;                      // at most; four of full tiles
constexpr int kSumWarps = 16, kWidth = 64;      // columns of a sum warp
constexpr int kThreads = 128 + 32 * kSumWarps;
constexpr int kChunk = 32 * kWidth * 2;         // a sum warp's output
constexpr int kTmem = 512;                      // two accumulators
constexpr int kScales = 6;                      // stages whose scales are made ahead
constexpr int kInfos = 16;                      // more tiles than warp 3 may be ahead of a sum: kScales and two loads
constexpr int kBars = (2 * kStages + 2 * kScales + 3) * 8 + 16;
constexpr int kSmem = 1024 + kRing + kSumWarps * kChunk + kScales * 1024 + kInfos * 16 + kBars + 2 * (kMaxExperts + 1) * 4;
static_assert(kSmem <= 227 * 1024, "shared memory");

struct Maps {
    CUtensorMap rows[8];  // [i]: one block of 16 (i + 1) rows
    CUtensorMap weight;   // forward: 128 rows of W; gradient: 128 columns
    CUtensorMap out;
};

struct Args {
    const int32_t *offsets;
    const float *row_scales, *weight_scales;
    const __nv_bfloat16 *bias;
    __nv_bfloat16 *out;
    int32_t *status;
    int32_t T, E;
    int32_t cols, depth;  // of the product
    int32_t zero_rest;
    int32_t scale_stride;  // of row_scales
    uint64_t timeout_ns;
};

struct Tile {
    int e, c0;            // expert, first column
    int r0, half, valid;  // first row, rows a CTA, rows that exist
};

struct Tiles {
    const int32_t *off, *start;
    int E, cols;

    __device__ __forceinline__ Tile at(int t) const
    {
        Tile x;
        x.e = expert_of(start, E, t);
        const int first = off[x.e], own = off[x.e + 1] - first;
        int ri, ci, r0, n;
        tile_place(t - start[x.e], (own + kBR - 1) / kBR, (cols + kBC - 1) / kBC, ri, ci);
        row_tile(own, kBR, kStep, ri, r0, n);
        x.c0 = ci * kBC;
        x.half = n / 2;
        x.valid = own - r0 < n ? own - r0 : n;
        x.r0 = first + r0;
        return x;
    }
};

__device__ __forceinline__ uint8_t *align1024(uint8_t *p)
{
    return reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

// Instruction descriptor, kind::f8f6f4: e4m3 A and B, fp32 D, shape M x N.
__device__ __forceinline__ constexpr uint32_t make_idesc_e4m3(int M, int N, bool b_mn)
{
    return (1u << 4)                                 // D format: f32
           | (static_cast<uint32_t>(b_mn) << 16)     // B major
           | (static_cast<uint32_t>(N >> 3) << 17)   // N / 8
           | (static_cast<uint32_t>(M >> 4) << 24);  // M / 16
}

__device__ __forceinline__ void umma_e4m3_lead_pair(uint32_t leader, uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi,
                                                    uint32_t b_lo, uint32_t b_hi, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 ad, bd;\n\t"
        "setp.ne.b32 e, %7, 0;\n\t"
        "mov.b64 ad, {%1, %2};\n\t"
        "mov.b64 bd, {%3, %4};\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], ad, bd, %5, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
}

// Two sums at a time: acc += v s.
__device__ __forceinline__ void fma2(uint64_t &acc, uint32_t v0, uint32_t v1, uint64_t s)
{
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(v0), "r"(v1));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(v), "l"(s));
}

__device__ __forceinline__ uint64_t twice(float s)
{
    uint64_t r;
    asm volatile("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(s));
    return r;
}

__device__ __forceinline__ float2 both(uint64_t v)
{
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}

// The scales of `n` blocks, up to four, that lie `step` apart, in whole 16 bytes if quads (n is 4 then); zero for the
// others, or if there are none.
__device__ __forceinline__ void load_scales(const float *at, int n, int64_t step, bool quads, bool exists, float (&s)[4])
{
    if (quads) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (exists) v = load_global(reinterpret_cast<const uint4 *>(at));
        s[0] = __uint_as_float(v.x), s[1] = __uint_as_float(v.y), s[2] = __uint_as_float(v.z), s[3] = __uint_as_float(v.w);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = exists && i < n ? load_float(at + i * step) : 0.f;
    }
}

// A warp's 32 rows x 64 columns, from column c on: sums, bias, one rounding, into shared memory (rows of 128 bytes,
// swizzled) and out by a copy, which takes its time while the next tile is summed; by plain stores where rows are
// missing: `rows` exist.
__device__ __forceinline__ void write_part(const Args &args, const CUtensorMap &map, uint8_t *buf, const uint64_t (&acc)[kWidth / 2],
                                           int e, int row0, int c, int rows, int lane)
{
    const __nv_bfloat16 *bias = args.bias ? args.bias + static_cast<int64_t>(e) * args.cols + c : nullptr;
    const int left = args.cols - c;  // a multiple of 8
    if (lane == 0) bulk_wait_group_read<0>();  // the tile before was read out
    __syncwarp();
#pragma unroll
    for (int j = 0; j < kWidth / 8; ++j) {
        uint4 bv = make_uint4(0, 0, 0, 0);
        if (bias && 8 * j < left) bv = load_global(reinterpret_cast<const uint4 *>(bias) + j);
        const uint32_t bw[4] = {bv.x, bv.y, bv.z, bv.w};
        uint32_t w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float2 f = both(acc[4 * j + u]);
            w[u] = pack_bf16x2(f.x + __uint_as_float(bw[u] << 16), f.y + __uint_as_float(bw[u] & 0xFFFF0000u));
        }
        *reinterpret_cast<uint4 *>(buf + lane * 128 + ((j ^ lane) & 7) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (rows >= 32) {
        fence_async_smem();
        __syncwarp();
        if (lane == 0) tma_store_3d(&map, buf, c, row0, 0);
    } else {
        __syncwarp();
        const int j = lane & 7;
        for (int r = lane >> 3; r < rows; r += 4)
            if (8 * j < left)
                *reinterpret_cast<uint4 *>(args.out + static_cast<int64_t>(row0 + r) * args.cols + c + 8 * j) =
                    *reinterpret_cast<const uint4 *>(buf + r * 128 + ((j ^ r) & 7) * 16);
        __syncwarp();
    }
    if (lane == 0) bulk_commit_group();  // one group a tile, an empty one for plain stores
}

__device__ __forceinline__ void named_bar_arrive(uint32_t id, uint32_t count)
{
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory");
}

// mbar_wait for a phase that is stages away: looks every 200 ns instead of sleeping inside try_wait, which polls shared
// memory (input gradient of 8192 rows, eight experts of 14336 x 4096: 557 us, 568 with mbar_wait; forward the same).
__device__ __forceinline__ bool wait_slowly(uint64_t *bar, uint32_t parity, uint64_t timeout_ns, const volatile int *abort)
{
    const uint32_t a = smem_u32(bar);
    if (mbar_test_wait(a, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (true) {
        __nanosleep(200);
        if (mbar_test_wait(a, parity)) return true;
        if (*abort || globaltimer_ns() - t0 > timeout_ns) return false;
    }
}

// An accumulator was read out and the stage's scales were read, as far as this warp reads them: `scales`, of this CTA, is
// released, so that those reads come before the slot is written again.
__device__ __forceinline__ void release(uint32_t bar, uint64_t *scales, int lane)
{
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
        mbar_arrive_cluster(bar);
        mbar_arrive(scales);
    }
}

// Bytes of a stage: a CTA's rows are half of the launch's largest tile.
__device__ __forceinline__ int stage_bytes(const int32_t *off, int32_t E)
{
    int top = 1;
    for (int e = threadIdx.x & 31; e < E; e += 32) top = max(top, off[e + 1] - off[e]);
    top = __reduce_max_sync(0xffffffffu, top);
    const int rows = top > kBR ? kBR : (top + kStep - 1) / kStep * kStep;
    return kWBytes + rows / 2 * kBlock;
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

template <bool kGrad>
__global__ void __launch_bounds__(kThreads, 1) k_fp8(const __grid_constant__ Maps maps, const Args args)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *stages = align1024(smem_raw);
    uint8_t *chunks = stages + kRing;  // 1024-byte aligned, as the swizzle wants
    float *scales = reinterpret_cast<float *>(chunks + kSumWarps * kChunk);      // [kScales][2][128]
    int4 *infos = reinterpret_cast<int4 *>(scales + kScales * 256);
    uint64_t *full = reinterpret_cast<uint64_t *>(infos + kInfos);  // copies of a stage landed (leader)
    uint64_t *empty = full + kStages;   // MMAs of a stage finished (each CTA)
    uint64_t *aempty = empty + kStages; // an accumulator was read out (leader)
    uint64_t *ready = aempty + 2;       // a stage's scales are there
    uint64_t *sfree = ready + kScales;  // ... were read by every sum warp
    uint64_t *drain = sfree + kScales;
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
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) mbar_init(&aempty[a], 2 * kSumWarps);
        for (int s = 0; s < kScales; ++s) {
            mbar_init(&ready[s], 1);
            mbar_init(&sfree[s], kSumWarps);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_map(&maps.weight);
        tma_prefetch_map(&maps.out);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, kTmem);
        tmem_relinquish_pair();
    }
    wait_for_prior_grid();  // nothing above touched global memory
    fetch_offsets(args.offsets, args.E, args.T, off);
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        clamp_offsets(args.E, args.T, off, args.status);
        const int nc = (args.cols + kBC - 1) / kBC;
        tile_starts(args.E, start, [&](int e) { return (off[e + 1] - off[e] + kBR - 1) / kBR * nc; });
        const int bytes = stage_bytes(off, args.E);
        if (lane == 0) *ring_slot = bytes;
    }
    __syncthreads();
    cluster_sync_all();  // the peer's barriers are initialised
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const Tiles tiles = {off, start, args.E, args.cols};
    const int count = start[args.E];
    const int first = blockIdx.x / 2, stride = gridDim.x / 2;
    const int stage = *ring_slot, S = kRing / stage < kStages ? kRing / stage : kStages;
    const int blocks = (args.depth + kBlock - 1) / kBlock;

    if (warp < 4) {
        if (warp == 0) {
            // ------------------------------------------------------------ producer: copies of the rows and of the weight
            if (lane == 0) {
                bool ok = true;
                int g = 0;  // stages issued
                Place at;
                for (int t = first; ok && t < count; t += stride) {
                    const Tile x = tiles.at(t);
                    const int row = x.r0 + static_cast<int>(rank) * x.half, col = x.c0 + static_cast<int>(rank) * 128;
                    const CUtensorMap *map = &maps.rows[x.half / 16 - 1];
                    const uint32_t bytes = 2 * (kWBytes + x.half * kBlock);
                    for (int b = 0; b < blocks; ++b, ++g, at.next(S)) {
                        if (g >= S && !mbar_wait(&empty[at.slot], at.parity ^ 1, tmo, abort_flag)) {
                            ok = false;
                            break;
                        }
                        uint8_t *dst = stages + at.slot * stage;
                        if (rank == 0) mbar_arrive_expect_tx(&full[at.slot], bytes);
                        const uint32_t bar = cluster_addr(&full[at.slot], 0);
                        // (maps count two-byte columns: 64 are a block)
                        if (kGrad) tma_load_3d_pair(dst, &maps.weight, bar, col / 2, b * kBlock, x.e);
                        else tma_load_3d_pair(dst, &maps.weight, bar, b * 64, col, x.e);
                        tma_load_3d_pair(dst + kWBytes, map, bar, b * 64, row, 0);
                    }
                }
                if (!ok) {
                    *abort_flag = 1;
                    set_status(args.status, BSL_ERR_TIMEOUT);
                } else {  // the MMAs' arrivals on this CTA's barriers are in
                    for (int s = 0; s < S && s < g; ++s) {
                        const int fills = (g - s + S - 1) / S;
                        if (!mbar_wait(&empty[s], (fills - 1) & 1, tmo, abort_flag)) set_status(args.status, BSL_ERR_TIMEOUT);
                    }
                }
                // every copy lands before shared memory is released: the last fill of
                // each slot is the newest phase of its barrier, which the leader holds
                if (rank == 0)
                    for (int s = 0; s < S && s < g; ++s) {
                        const int fills = (g - s + S - 1) / S;
                        if (!mbar_wait(&full[s], (fills - 1) & 1, tmo, nullptr)) set_status(args.status, BSL_ERR_TIMEOUT);
                    }
            }
            __syncwarp();
        } else if (warp == 1) {
            // ------------------------------------------------------------ MMA issuer (the leader's)
            // What a stage costs this warp is time that the tensor pipe may stand idle, so the loop is flat and one commit
            // tells the producers and the sums.
            if (rank == 0) {
                const uint32_t lead = lane == 0;
                // (the same in all lanes, and said so: an MMA's operands stay in uniform registers)
                const uint32_t tm = uniform(tmem), bytes = uniform(static_cast<uint32_t>(stage));
                const int ring = uniform(S), total = uniform(count > first ? (count - first + stride - 1) / stride * blocks : 0);
                const uint32_t idesc = make_idesc_e4m3(256, kBC, kGrad);
                // K-major: 8-row atoms 1024 bytes apart, a K step of 32 bytes along the row; N-major: atoms of
                // 8 rows 1024 bytes apart, a K step of 32 rows of 128 bytes
                const uint64_t desc = make_sdesc(smem_u32(stages), 16, 1024, kLayoutSw128);
                const uint32_t base = uniform(static_cast<uint32_t>(desc)), hi = uniform(static_cast<uint32_t>(desc >> 32));
                bool ok = true;
                Place at;
                for (int it = 0; it < total; ++it) {
                    const int acc = it & 1;
                    if (!mbar_wait(&full[at.slot], at.parity, tmo, abort_flag) ||
                        (it >= 2 && !mbar_wait(&aempty[acc], ((it >> 1) - 1) & 1, tmo, abort_flag)))
                        ok = false;
                    if (__any_sync(0xffffffffu, !ok)) break;
                    tc_fence_after();
                    const uint32_t blo = base + at.slot * (bytes >> 4), alo = blo + (kWBytes >> 4);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        umma_e4m3_lead_pair(lead, tm + acc * kBC, alo + 2 * i, hi, blo + (kGrad ? 256 : 2) * i, hi, idesc, i != 0);
                    umma_commit_lead_pair(lead, &empty[at.slot]);
                    at.next(ring);
                }
                ok = !__any_sync(0xffffffffu, !ok);
                if (lane == 0 && !ok) {
                    *abort_flag = 1;
                    set_status(args.status, BSL_ERR_TIMEOUT);
                }
                // every MMA is complete before TMEM and shared memory are released
                umma_commit_lead_pair(lead, drain);
                if (lane == 0 && !mbar_wait(drain, 0, tmo, nullptr)) set_status(args.status, BSL_ERR_TIMEOUT);
            }
            __syncwarp();
        } else {
            const int total = count > first ? (count - first + stride - 1) / stride * blocks : 0;
            bool ok = true;
            if (warp == 2) {
                // ---------------------------------------------------- the wait for the MMAs of a stage, for the sums
                Place at, sc;
                for (int it = 0; it < total; ++it, at.next(S), sc.next(kScales)) {
                    if (ok && (__any_sync(0xffffffffu, !mbar_wait(&empty[at.slot], at.parity, tmo, abort_flag)) ||
                               __any_sync(0xffffffffu, !mbar_wait(&ready[sc.slot], sc.parity, tmo, abort_flag)))) {
                        ok = false;
                        if (lane == 0) *abort_flag = 1;
                        __syncwarp();
                    }
                    if (ok) named_bar_arrive(1 + (it & 1), 32 * kSumWarps + 32);
                    else named_bar_sync(1 + (it & 1), 32 * kSumWarps + 32);  // an aborted run's sums go on to the end, in step
                }
            } else {
                // ---------------------------------------------------- scales
                const int wide_blocks = (args.cols + 127) / 128;
                const int64_t plane = static_cast<int64_t>(wide_blocks) * blocks, wstep = kGrad ? wide_blocks : 1;
                // what is loaded next: tile, block, and what is known of the tile
                int t = first, b = 0, n = 0, rows = 0;
                const float *rs = nullptr, *ws = nullptr;
                bool second = false;
                const bool quads = args.scale_stride % 4 == 0, wquads = !kGrad && blocks % 4 == 0;
                struct Four {  // blocks' scales: of this lane's rows 32 apart, and of the weight's two tiles
                    float row[4][4], col[2][4];
                    int n;
                };
                auto load = [&](Four &f) {
                    f.n = 0;
                    if (t >= count) return;
                    if (b == 0) {
                        const Tile x = tiles.at(t);
                        const int in_tile = static_cast<int>(rank) * x.half;
                        rows = max(0, min(x.half, x.valid - in_tile));
                        if (lane == 0) infos[n % kInfos] = make_int4(x.e, x.c0, x.r0 + in_tile, rows);
                        rs = args.row_scales + (static_cast<int64_t>(x.r0) + in_tile + lane) * args.scale_stride;
                        ws = args.weight_scales + x.e * plane + x.c0 / 128 * (kGrad ? 1 : static_cast<int64_t>(blocks));
                        second = x.c0 + 128 < args.cols;
                    }
                    f.n = min(4, blocks - b);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        load_scales(rs + 32 * i * static_cast<int64_t>(args.scale_stride) + b, f.n, 1, quads, lane + 32 * i < rows,
                                    f.row[i]);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        load_scales(ws + i * (kGrad ? 1 : static_cast<int64_t>(blocks)) + b * wstep, f.n, wstep, wquads, !i || second,
                                    f.col[i]);
                    if ((b += f.n) == blocks) b = 0, t += stride, ++n;
                };
                int made = 0;
                auto make = [&](const Four &f) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (!ok || j >= f.n) break;
                        // where stage made - kScales was, whose scales every sum warp has read
                        const int round = made / kScales, slot = made - round * kScales;
                        if (round > 0) ok = __all_sync(0xffffffffu, wait_slowly(&sfree[slot], (round - 1) & 1, tmo, abort_flag));
                        if (!ok) break;
                        float *to = scales + slot * 256 + lane;
#pragma unroll
                        for (int i = 0; i < 4; ++i) to[32 * i] = f.row[i][j] * f.col[0][j], to[128 + 32 * i] = f.row[i][j] * f.col[1][j];
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&ready[slot]);
                        ++made;
                    }
                };
                // two sets of four blocks in turn: one's loads have the other's stages to arrive
                Four f, g;
                load(f);
                load(g);
                while (ok && made < total) {
                    make(f);
                    load(f);
                    make(g);
                    load(g);
                }
                if (args.zero_rest) {  // rows of no expert
                    zero_range(args.out, 0, static_cast<int64_t>(off[0]) * args.cols, lane);
                    zero_range(args.out, static_cast<int64_t>(off[args.E]) * args.cols, static_cast<int64_t>(args.T) * args.cols,
                               lane);
                }
            }
            if (lane == 0 && !ok) {
                *abort_flag = 1;
                set_status(args.status, BSL_ERR_TIMEOUT);
            }
            __syncwarp();
        }
    } else {
        // ------------------------------------------------------------ sums
        const int q = warp & 3, part = (warp - 4) >> 2;
        const uint32_t mine = tmem + (static_cast<uint32_t>(32 * q) << 16) + part * kWidth;
        uint8_t *chunk = chunks + (warp - 4) * kChunk;
        const float *my_scales = scales + part / 2 * 128 + 32 * q + lane;
        bool ok = true;
        int it = 0, ring = 0, n = 0;
        for (int t = first; t < count; t += stride, ++n) {
            uint64_t acc[kWidth / 2];
#pragma unroll
            for (int i = 0; i < kWidth / 2; ++i) acc[i] = 0;
            bool live = false;
#pragma unroll 1
            for (int b = 0; b < blocks; ++b, ++it) {
                const int buf = it & 1;
                named_bar_sync(1 + buf, 32 * kSumWarps + 32);
                tc_fence_after();
                if (b == 0) live = infos[n % kInfos].w > 32 * q && infos[n % kInfos].y + kWidth * part < args.cols;
                const uint64_t s2 = twice(my_scales[ring * 256]);
                if (live) {
                    const uint32_t from = mine + buf * kBC;
                    uint32_t v[2][16];
                    tmem_ld16(from, v[0]);
#pragma unroll
                    for (int j = 0; j < kWidth / 16; ++j) {
                        tmem_wait_ld();
                        if (j + 1 < kWidth / 16) tmem_ld16(from + 16 * (j + 1), v[(j + 1) & 1]);
                        else release(cluster_addr(&aempty[buf], 0), &sfree[ring], lane);
#pragma unroll
                        for (int u = 0; u < 8; ++u) fma2(acc[8 * j + u], v[j & 1][2 * u], v[j & 1][2 * u + 1], s2);
                    }
                } else {
                    release(cluster_addr(&aempty[buf], 0), &sfree[ring], lane);
                }
                if (++ring == kScales) ring = 0;
            }
            if (*abort_flag) ok = false;
            if (ok && live) {
                const int4 x = infos[n % kInfos];  // expert, first column, first row, rows
                write_part(args, maps.out, chunk, acc, x.x, x.z + 32 * q, x.y + kWidth * part, x.w - 32 * q, lane);
            }
            __syncwarp();
        }
        if (lane == 0) bulk_wait_group<0>();
        if (lane == 0 && !ok) {
            *abort_flag = 1;
            set_status(args.status, BSL_ERR_TIMEOUT);
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
        tmem_dealloc_pair(tmem, kTmem);
    }
}

template <bool kGrad>
bsl_status run(const Maps &maps, const Args &args, cudaStream_t s)
{
    auto kern = k_fp8<kGrad>;
    const bsl_status sa = set_smem_once(reinterpret_cast<const void *>(kern), kSmem);
    if (sa != BSL_OK) return sa;
    return cuda_status(launch_dependent_cluster(kern, num_sms() / 2 * 2, 2, kThreads, kSmem, s, maps, args));
}

}  // namespace

bsl_status launch_fp8(const uint8_t *codes, const float *scales, int32_t T, const int32_t *offsets, const bsl_fp8 *W,
                      bool transposed, const void *bias, void *out, int32_t zero_rest, bool early, cudaStream_t s)
{
    if (!transposed && few_rows8(T)) return launch_few_rows8(codes, scales, T, offsets, W, bias, out, zero_rest, s);
    if (fp8_few(T, W->E, transposed ? W->K : W->N))
        return launch_fp8_few(codes, scales, T, offsets, W, transposed, bias, out, zero_rest, early, s);
    Args args = {};
    args.offsets = offsets;
    args.row_scales = scales;
    args.weight_scales = W->scales;
    args.bias = static_cast<const __nv_bfloat16 *>(bias);
    args.out = static_cast<__nv_bfloat16 *>(out);
    args.status = W->status;
    args.T = T;
    args.E = W->E;
    args.cols = transposed ? W->K : W->N;
    args.depth = transposed ? W->N : W->K;
    args.zero_rest = zero_rest;
    args.scale_stride = (args.depth + 127) / 128;
    args.timeout_ns = wait_timeout_ns();
    Maps m;
    const int64_t K = W->K, N = W->N;
    bool good = make_map_3d(&m.weight, W->codes, K / 2, N, W->E, K, K * N, 64, 128, 128) &&
                make_map_3d(&m.out, out, args.cols, T, 1, static_cast<uint64_t>(args.cols) * 2,
                            static_cast<uint64_t>(args.cols) * 2 * T, kWidth, 32, 128);
    // (a CTA has no more than T rows, rounded up to 16)
    for (int i = 0; i < 8 && 16 * i < T; ++i)
        good = good && make_map_3d(&m.rows[i], codes, args.depth / 2, T, 1, args.depth,
                                   static_cast<uint64_t>(args.depth) * T, 64, 16 * (i + 1), 128);
    if (!good) return BSL_ERR_CUDA;
    return transposed ? run<true>(m, args, s) : run<false>(m, args, s);
}

}  // namespace bsl
