// fp8.cu -- products of 8-bit (e4m3) matrices with a scale for each block of 128
// (fp8_quant.cu gives the format), dense or grouped by expert:
//     forward          Y[t][n]  = sum_b sx[t][b] sw[n/128][b] sum_{k in b} x[t][k] w[n][k] (+ bias)
//     input gradient   dX[t][k] = sum_b sg[t][b] sw[b][k/128] sum_{n in b} g[t][n] w[n][k]
//
// The scales are fp32 numbers, which the tensor cores do not take, and change
// every 128 elements of the sum.  So each block's sum is an accumulator of its
// own in TMEM, and eight warps bring it to registers, multiply it by the two
// scales and add it to the output's sum there, 32 bits throughout, while the
// MMAs fill the other accumulator.  The rows t go to the MMA's M side, the
// TMEM lanes: a lane's scale is then one number per thread and block, and the
// weight's is one per warp (its 128 columns are one tile of the weight), so
// a block costs a thread one FMA per column.  With the features on the lanes, as
// in the bf16 kernel, every column would need a scale of its own from shared
// memory: four times the bytes of the sum itself.
//
// Clusters of two CTAs work on tiles of up to 256 rows x 256 columns
// (cta_group::2, M = 256): each CTA holds half of the tile's rows, its 128 lanes,
// and half of the weight's columns.  A stage is one block: 16 KB of each
// operand, at 512 clocks of MMA, 256 of FMA and 256 of TMEM reads.  An
// expert's rows are spread evenly over the fewest tiles, and copies bring
// exactly a tile's rows.  The weight is K-major in the forward and N-major
// in the gradient, the same codes for both.
//
// Persistent kernels, programmatic dependents, 12 warps a CTA:
//   warps 0, 2  TMA producers of the rows and of the weight (a ring of stages);
//   warp 1      MMA issuer and TMEM owner;
//   warp 3      zeros for the rows of no expert, on request;
//   warps 4-11  sums: TMEM -> registers; warp 4 + 4g + q owns lanes 32q .. of
//               columns 128g .. and holds their 128 x 32 sums in 128 registers a
//               thread (setmaxnreg: 216 for these, 72 for the others).
// A tile's output goes from registers to global memory in whole sectors, 32
// bytes a lane.  Tiles are dealt round robin; no workspace is shared by
// calls, and every output is one sum in a fixed order.
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
constexpr int kRing = 192 * 1024;
constexpr int kStages = 12;                     // at most
constexpr int kSumWarps = 8;
constexpr int kThreads = 128 + 32 * kSumWarps;
constexpr int kTmem = 512;                      // two accumulators
constexpr int kBars = (2 * kStages + 5) * 8 + 16;
constexpr int kSmem = 1024 + kRing + kBars + 2 * (kMaxExperts + 1) * 4;
static_assert(kSmem <= 227 * 1024, "shared memory");
// setmaxnreg moves registers inside the block's own: 384 threads x 168
constexpr int kLaunchRegs = 168, kSumRegs = 216, kOtherRegs = 72;
static_assert(32 * kSumWarps * kSumRegs + 128 * kOtherRegs <= kThreads * kLaunchRegs, "registers");

struct Maps {
    CUtensorMap rows[8];  // [i]: one block of 16 (i + 1) rows
    CUtensorMap weight;   // forward: 128 rows of W; gradient: 128 columns
};

struct Args {
    const int32_t *offsets;
    const float *row_scales, *weight_scales;
    const __nv_bfloat16 *bias;
    __nv_bfloat16 *out;
    int32_t *status;
    int32_t T, E;
    int32_t cols, depth;  // of the product
    int32_t zero_rest, wide;  // wide: 32-byte stores may be used
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

template <int kRegs>
__device__ __forceinline__ void more_registers()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}

template <int kRegs>
__device__ __forceinline__ void fewer_registers()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
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
    asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(s));
    return r;
}

__device__ __forceinline__ float2 both(uint64_t v)
{
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}

// The scales of four blocks b .. b + 3 of a row (of `count` blocks `step` apart); past the end: zero.
__device__ __forceinline__ void load_scales(const float *row, int b, int count, int64_t step, bool vec, bool exists,
                                            float (&s)[4])
{
    if (vec && exists && b < count) {
        const uint4 v = load_global(reinterpret_cast<const uint4 *>(row + b));
        s[0] = __uint_as_float(v.x), s[1] = __uint_as_float(v.y), s[2] = __uint_as_float(v.z), s[3] = __uint_as_float(v.w);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = exists && b + i < count ? load_float(row + (b + i) * step) : 0.f;
}

// 128 columns of a row, from column c on: sums, bias, one rounding, whole sectors.
__device__ __forceinline__ void write_row(const Args &args, const uint64_t (&acc)[64], int e, int64_t row, int c)
{
    __nv_bfloat16 *out = args.out + row * args.cols + c;
    const __nv_bfloat16 *bias = args.bias ? args.bias + static_cast<int64_t>(e) * args.cols + c : nullptr;
    const int left = args.cols - c;  // a multiple of 8
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        uint32_t w[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint4 bv = make_uint4(0, 0, 0, 0);
            if (bias && 16 * j + 8 * h < left) bv = load_global(reinterpret_cast<const uint4 *>(bias + 16 * j + 8 * h));
            const uint32_t bw[4] = {bv.x, bv.y, bv.z, bv.w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                float2 f = both(acc[8 * j + 4 * h + u]);
                if (bias) f.x += __uint_as_float(bw[u] << 16), f.y += __uint_as_float(bw[u] & 0xFFFF0000u);
                w[4 * h + u] = pack_bf16x2(f.x, f.y);
            }
        }
        __nv_bfloat16 *to = out + 16 * j;
        if (args.wide && 16 * j + 16 <= left) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                             __cvta_generic_to_global(to)),
                         "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                         : "memory");
        } else {
            if (16 * j < left) *reinterpret_cast<uint4 *>(to) = make_uint4(w[0], w[1], w[2], w[3]);
            if (16 * j + 8 < left) *reinterpret_cast<uint4 *>(to + 8) = make_uint4(w[4], w[5], w[6], w[7]);
        }
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
    uint64_t *full = reinterpret_cast<uint64_t *>(stages + kRing);  // copies of a stage landed (leader)
    uint64_t *empty = full + kStages;                               // MMAs of a stage finished (each CTA)
    uint64_t *afull = empty + kStages;                              // a block's sum complete (each CTA)
    uint64_t *aempty = afull + 2;                                   // ... read out (leader)
    uint64_t *drain = aempty + 2;
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
        for (int a = 0; a < 2; ++a) {
            mbar_init(&afull[a], 1);
            mbar_init(&aempty[a], 2 * kSumWarps);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_map(&maps.weight);
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
        fewer_registers<kOtherRegs>();
        if (warp == 0 || warp == 2) {
            // -------------------------------------------------------- producers: warp 0 copies rows, warp 2 the weight
            if (lane == 0) {
                const bool is_a = warp == 0;
                bool ok = true;
                int g = 0;  // stages issued
                Place at;
                for (int t = first; ok && t < count; t += stride) {
                    const Tile x = tiles.at(t);
                    const int row = x.r0 + static_cast<int>(rank) * x.half, col = x.c0 + static_cast<int>(rank) * 128;
                    const CUtensorMap *map = is_a ? &maps.rows[x.half / 16 - 1] : &maps.weight;
                    const uint32_t bytes = 2 * (kWBytes + x.half * kBlock);
                    for (int b = 0; b < blocks; ++b, ++g, at.next(S)) {
                        if (g >= S && !mbar_wait(&empty[at.slot], at.parity ^ 1, tmo, abort_flag)) {
                            ok = false;
                            break;
                        }
                        uint8_t *dst = stages + at.slot * stage + (is_a ? kWBytes : 0);
                        if (is_a && rank == 0) mbar_arrive_expect_tx(&full[at.slot], bytes);
                        const uint32_t bar = cluster_addr(&full[at.slot], 0);
                        // (maps count two-byte columns: 64 are a block)
                        if (is_a) tma_load_3d_pair(dst, map, bar, b * 64, row, 0);
                        else if (kGrad) tma_load_3d_pair(dst, map, bar, col / 2, b * kBlock, x.e);
                        else tma_load_3d_pair(dst, map, bar, b * 64, col, x.e);
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
            // -------------------------------------------------------- MMA issuer (the leader's)
            if (rank == 0) {
                const uint32_t lead = lane == 0;
                // (the same in all lanes, and said so: an MMA's operands stay in uniform registers)
                const uint32_t tm = uniform(tmem);
                const int tiles_end = uniform(count), ring = uniform(S);
                const uint32_t bytes = uniform(static_cast<uint32_t>(stage));
                const uint32_t idesc = make_idesc_e4m3(256, kBC, kGrad);
                bool ok = true;
                Place at;
                int it = 0;  // blocks so far
                for (int t = first; ok && t < tiles_end; t += stride) {
                    for (int b = 0; b < blocks; ++b, ++it, at.next(ring)) {
                        const int acc = it & 1;
                        if (__any_sync(0xffffffffu, !mbar_wait(&full[at.slot], at.parity, tmo, abort_flag)) ||
                            (it >= 2 &&
                             __any_sync(0xffffffffu, !mbar_wait(&aempty[acc], ((it >> 1) - 1) & 1, tmo, abort_flag)))) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t b0 = smem_u32(stages) + at.slot * bytes, a0 = b0 + kWBytes;
                        // K-major: 8-row atoms 1024 bytes apart, a K step of 32 bytes along the row; N-major: atoms of
                        // 8 rows 1024 bytes apart, a K step of 32 rows of 128 bytes
                        const uint64_t ad = make_sdesc(a0, 16, 1024, kLayoutSw128);
                        const uint64_t bd = make_sdesc(b0, 16, 1024, kLayoutSw128);
                        const uint32_t alo = static_cast<uint32_t>(ad), ahi = static_cast<uint32_t>(ad >> 32);
                        const uint32_t blo = static_cast<uint32_t>(bd), bhi = static_cast<uint32_t>(bd >> 32);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            umma_e4m3_lead_pair(lead, tm + acc * kBC, alo + 2 * i, ahi, blo + (kGrad ? 256 : 2) * i, bhi, idesc,
                                                i != 0);
                        umma_commit_lead_pair(lead, &empty[at.slot]);
                        umma_commit_lead_pair(lead, &afull[acc]);
                        __syncwarp();
                    }
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
        } else {
            // -------------------------------------------------------- rows of no expert
            if (args.zero_rest) {
                zero_range(args.out, 0, static_cast<int64_t>(off[0]) * args.cols, lane);
                zero_range(args.out, static_cast<int64_t>(off[args.E]) * args.cols,
                           static_cast<int64_t>(args.T) * args.cols, lane);
            }
            __syncwarp();
        }
    } else {
        // ------------------------------------------------------------ sums
        more_registers<kSumRegs>();
        const int q = warp & 3, part = (warp - 4) >> 2;
        const uint32_t mine = tmem + (static_cast<uint32_t>(32 * q) << 16) + part * 128;
        const int wide_blocks = (args.cols + 127) / 128;                   // tiles of the weight along the columns
        const int64_t plane = static_cast<int64_t>(wide_blocks) * blocks;  // its scales
        const bool vec = blocks % 4 == 0;
        bool ok = true;
        int it = 0;
        for (int t = first; ok && t < count; t += stride) {
            const Tile x = tiles.at(t);
            const int c = x.c0 + 128 * part, lrow = 32 * q + lane, in_tile = static_cast<int>(rank) * x.half + lrow;
            const bool exists = lrow < x.half && in_tile < x.valid && c < args.cols;
            const int64_t row = x.r0 + in_tile;
            const bool any = c < args.cols && 32 * q < x.half && static_cast<int>(rank) * x.half + 32 * q < x.valid;
            const float *rs = args.row_scales + row * blocks;
            const float *ws = args.weight_scales + x.e * plane + (kGrad ? c / 128 : static_cast<int64_t>(c / 128) * blocks);
            uint64_t acc[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = 0;
            float sr[4], sw[4];
            load_scales(rs, 0, blocks, 1, vec, exists, sr);
            load_scales(ws, 0, blocks, kGrad ? wide_blocks : 1, !kGrad && vec, any, sw);
            for (int b0 = 0; ok && b0 < blocks; b0 += 4) {
                float s[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) s[i] = sr[i] * sw[i];
                load_scales(rs, b0 + 4, blocks, 1, vec, exists, sr);
                load_scales(ws, b0 + 4, blocks, kGrad ? wide_blocks : 1, !kGrad && vec, any, sw);
#pragma unroll 1
                for (int i = 0; i < 4 && b0 + i < blocks; ++i, ++it) {
                    const int buf = it & 1;
                    const uint64_t s2 = twice(s[0]);
                    s[0] = s[1], s[1] = s[2], s[2] = s[3];
                    if (__any_sync(0xffffffffu, !mbar_wait(&afull[buf], (it >> 1) & 1, tmo, abort_flag))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (any) {
                        const uint32_t at = mine + buf * kBC;
                        uint32_t v[2][32];
                        tmem_ld32(at, v[0]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            tmem_wait_ld();
                            if (j < 3) tmem_ld32(at + 32 * (j + 1), v[(j + 1) & 1]);
                            else tc_fence_before();
#pragma unroll
                            for (int u = 0; u < 16; ++u) fma2(acc[16 * j + u], v[j & 1][2 * u], v[j & 1][2 * u + 1], s2);
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(cluster_addr(&aempty[buf], 0));
                }
            }
            if (ok && exists) write_row(args, acc, x.e, row, c);
            __syncwarp();
        }
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
    // the register split waits for ever if the block is launched with fewer than it adds up to
    static const int regs = [] {
        cudaFuncAttributes at = {};
        return cudaFuncGetAttributes(&at, k_fp8<kGrad>) == cudaSuccess ? at.numRegs : 0;
    }();
    if (regs < kLaunchRegs) return BSL_ERR_UNSUPPORTED;
    return cuda_status(launch_dependent_cluster(kern, num_sms() / 2 * 2, 2, kThreads, kSmem, s, maps, args));
}

}  // namespace

bsl_status launch_fp8(const uint8_t *codes, const float *scales, int32_t T, const int32_t *offsets, const bsl_fp8 *W,
                      bool transposed, const void *bias, void *out, int32_t zero_rest, cudaStream_t s)
{
    if (!transposed && few_rows8(T, W)) return launch_few_rows8(codes, scales, T, offsets, W, bias, out, zero_rest, s);
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
    args.wide = args.cols % 16 == 0 && reinterpret_cast<uintptr_t>(out) % 32 == 0;
    args.timeout_ns = wait_timeout_ns();
    Maps m;
    const int64_t K = W->K, N = W->N;
    bool good = make_map_3d(&m.weight, W->codes, K / 2, N, W->E, K, K * N, 64, 128, 128);
    // (a CTA has no more than T rows, rounded up to 16)
    for (int i = 0; i < 8 && 16 * i < T; ++i)
        good = good && make_map_3d(&m.rows[i], codes, args.depth / 2, T, 1, args.depth,
                                   static_cast<uint64_t>(args.depth) * T, 64, 16 * (i + 1), 128);
    if (!good) return BSL_ERR_CUDA;
    return transposed ? run<true>(m, args, s) : run<false>(m, args, s);
}

}  // namespace bsl
