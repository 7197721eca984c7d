// fp8_few.cu -- products of the 8-bit layer for tiles of few rows: the forward
// Y[t] = X[t] . W[e]^T + bias[e] and the input gradient dX[t] = dY[t] . W[e] (fp8.cu has the
// formulas with the scales, and the kernel for many rows).
//
// Reading the reached experts' weights once bounds it.  In the kernel for many
// rows a tile's sums take as long with few rows as with 128 a CTA, since they go by
// TMEM lanes.  Here the output's columns are on the MMA's M side, the lanes (the weight
// K-major, or M-major in the gradient), and up to 64 rows on its N side: a block's sum has a column for each row, whose scale comes from
// shared memory, already multiplied by the weight's (one tile of 128 features has one).
// mma.sync is no way out: its 8-bit form unpacks the codes by instructions, 300 for
// 2 KB of weight, and those bound it (64 rows of 16 experts of 11008 x 4096: 202 us,
// the kernel for many rows 188, this one 145; the bytes at the rate of a copy 110).
//
// One CTA an SM, 8 warps: 0 copies, 1 MMAs, 2 scales, 3 zeros for the rows of no
// expert, 4-7 sums (a thread has one column and all rows).  A stage is one block of
// 128, 16 KB of weight; sums wait for it in four accumulators.  Where tiles of 128
// columns are fewer than the SMs, the CTAs of a cluster cut the blocks and add up their sums
// through shared memory, in order.
//
// Every wait is bounded, as in fp8.cu.
#include "grouped.cuh"
#include "internal.h"
#include "pair.cuh"

namespace bsl {
namespace {

constexpr int kCols = 128, kMostRows = 64, kStep = 16;  // of a tile; granularity of the rows
constexpr int kBlock = 128;
constexpr int kWBytes = kCols * kBlock;
constexpr int kRing = 176 * 1024, kStages = 10;
constexpr int kAcc = 4, kTmem = kAcc * kMostRows;  // accumulators
constexpr int kScales = 8;                         // stages' scales
constexpr int kThreads = 256;
constexpr int kPartStride = kCols + 1;
constexpr int kPart = kMostRows * kPartStride * 4;  // a CTA's sums, in the ring's place
constexpr int kBars = (2 * kStages + 2 * kAcc + 2 * kScales + 1) * 8 + 16;
constexpr int kSmem = 1024 + kRing + kScales * kMostRows * 4 + kBars + 2 * (kMaxExperts + 1) * 4;
static_assert(kSmem <= 227 * 1024 && kPart <= kRing, "shared memory");

struct Maps {
    CUtensorMap weight;   // one tile of 128 x 128
    CUtensorMap rows[4];  // [i]: 16 (i + 1) rows of one block
};

struct Args {
    const int32_t *offsets;
    const float *row_scales, *weight_scales;
    const __nv_bfloat16 *bias;
    __nv_bfloat16 *out;
    int32_t *status;
    int32_t T, E;
    int32_t cols, depth;       // of the product
    int32_t zero_rest, early;  // early: the weight and the offsets are older than the kernel before
    int32_t parts;             // CTAs that cut the blocks
    uint64_t timeout_ns;
};

struct Tile {
    int e, c0, r0, rows, n;  // expert, first column, first row, rows, MMA N
};

struct Tiles {
    const int32_t *off, *start;
    int E;

    __device__ __forceinline__ Tile at(int t) const
    {
        Tile x;
        x.e = expert_of(start, E, t);
        const int first = off[x.e], own = off[x.e + 1] - first, groups = (own + kMostRows - 1) / kMostRows;
        const int i = t - start[x.e], c = i / groups;  // groups of one column tile side by side: the weight is in L2
        int r0, n;
        row_tile(own, kMostRows, kStep, i - c * groups, r0, n);
        x.c0 = c * kCols;
        x.n = n;
        x.rows = own - r0 < n ? own - r0 : n;
        x.r0 = first + r0;
        return x;
    }
};

// A place in a ring: slot, and the parity of the phase that fills it.
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

__device__ __forceinline__ void umma_e4m3_lead(uint32_t leader, uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t hi,
                                               uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 ad, bd;\n\t"
        "setp.ne.b32 e, %6, 0;\n\t"
        "mov.b64 ad, {%1, %3};\n\t"
        "mov.b64 bd, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], ad, bd, %4, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
}

template <bool kGrad>
__global__ void __launch_bounds__(kThreads, 1) k_fp8_few(const __grid_constant__ Maps maps, const Args args)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *stages = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *scales = reinterpret_cast<float *>(stages + kRing);       // [kScales][kMostRows]
    uint64_t *full = reinterpret_cast<uint64_t *>(scales + kScales * kMostRows);  // copies of a stage landed
    uint64_t *empty = full + kStages;    // MMAs of a stage done
    uint64_t *afull = empty + kStages;   // an accumulator complete
    uint64_t *aempty = afull + kAcc;     // ... read out
    uint64_t *sfull = aempty + kAcc;     // a stage's scales there
    uint64_t *sempty = sfull + kScales;  // ... used
    uint64_t *drain = sempty + kScales;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *ring_slot = reinterpret_cast<int *>(tmem_slot + 2);
    int32_t *off = reinterpret_cast<int32_t *>(tmem_slot + 4);
    int32_t *start = off + kMaxExperts + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int parts = args.parts, rank = blockIdx.x % parts;
    const uint64_t tmo = args.timeout_ns;
    dependents_may_launch();
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < kAcc; ++a) {
            mbar_init(&afull[a], 1);
            mbar_init(&aempty[a], 4);
        }
        for (int s = 0; s < kScales; ++s) {
            mbar_init(&sfull[s], 1);
            mbar_init(&sempty[s], 4);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_map(&maps.weight);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, kTmem);
        tmem_relinquish();
    }
    if (!args.early) wait_for_prior_grid();  // nothing above touched global memory
    fetch_offsets(args.offsets, args.E, args.T, off);
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        clamp_offsets(args.E, args.T, off, blockIdx.x == 0 ? args.status : nullptr);
        const int nc = (args.cols + kCols - 1) / kCols;
        tile_starts(args.E, start, [&](int e) { return (off[e + 1] - off[e] + kMostRows - 1) / kMostRows * nc; });
        int top = 1;
        for (int e = lane; e < args.E; e += 32) top = max(top, off[e + 1] - off[e]);
        top = __reduce_max_sync(0xffffffffu, top);
        const int rows = top > kMostRows ? kMostRows : (top + kStep - 1) / kStep * kStep;
        if (lane == 0) *ring_slot = kWBytes + rows * kBlock;
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const Tiles tiles = {off, start, args.E};
    const int count = start[args.E], first = blockIdx.x / parts, stride = gridDim.x / parts;
    const int stage = *ring_slot, S = kRing / stage < kStages ? kRing / stage : kStages;
    const int blocks = (args.depth + kBlock - 1) / kBlock;
    const int kb0 = static_cast<int>(static_cast<int64_t>(blocks) * rank / parts);
    const int own = static_cast<int>(static_cast<int64_t>(blocks) * (rank + 1) / parts) - kb0;  // blocks of this CTA
    const int total = count > first ? (count - first + stride - 1) / stride * own : 0;
    bool ok = true;

    if (warp == 0) {
        // ------------------------------------------------------------ copies
        if (lane == 0) {
            auto copy_weight = [&](const Tile &x, int b, int slot) {  // (maps count two-byte columns: 64 are a block)
                uint8_t *dst = stages + slot * stage;
                if (kGrad) tma_load_3d(dst, &maps.weight, &full[slot], x.c0 / 2, (kb0 + b) * kBlock, x.e);
                else tma_load_3d(dst, &maps.weight, &full[slot], (kb0 + b) * 64, x.c0, x.e);
            };
            int g = 0;
            Place at;
            // what is older than the kernel before may be copied before the wait for it: the weight's first stages
            int ahead = 0;
            if (args.early) {
                if (total > 0) {
                    const Tile x = tiles.at(first);
                    for (; ahead < S && ahead < own; ++ahead) copy_weight(x, ahead, ahead);
                }
                wait_for_prior_grid();
            }
            for (int t = first; ok && t < count; t += stride) {
                const Tile x = tiles.at(t);
                const uint32_t bytes = kWBytes + x.n * kBlock;
                for (int b = 0; b < own; ++b, ++g, at.next(S)) {
                    if (g >= S && !mbar_wait(&empty[at.slot], at.parity ^ 1, tmo, abort_flag)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&full[at.slot], bytes);
                    if (g >= ahead) copy_weight(x, b, at.slot);
                    tma_load_3d(stages + at.slot * stage + kWBytes, &maps.rows[x.n / kStep - 1], &full[at.slot], (kb0 + b) * 64, x.r0, 0);
                }
            }
            // every copy lands before shared memory is released: the last fill of each slot is its barrier's newest phase
            for (int s = 0; s < S && s < g; ++s)
                if (!mbar_wait(&full[s], ((g - s + S - 1) / S - 1) & 1, tmo, nullptr)) ok = false;
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMAs
        const uint32_t lead = lane == 0;
        const uint32_t tm = uniform(tmem), bytes = uniform(static_cast<uint32_t>(stage));
        const uint64_t desc = make_sdesc(smem_u32(stages), 16, 1024, kLayoutSw128);  // atoms of 8 rows 1024 bytes apart
        const uint32_t base = uniform(static_cast<uint32_t>(desc)), hi = uniform(static_cast<uint32_t>(desc >> 32));
        Place at, acc;
        int it = 0;
        for (int t = first; ok && t < count; t += stride) {
            const int n = uniform(tiles.at(t).n);
            // kind::f8f6f4: fp32 D, e4m3 A and B, A's major, N / 8, M / 16
            const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(kGrad) << 15) | (static_cast<uint32_t>(n >> 3) << 17) |
                                   (static_cast<uint32_t>(kCols >> 4) << 24);
            for (int b = 0; b < own; ++b, ++it, at.next(S), acc.next(kAcc)) {
                if (__any_sync(0xffffffffu, !mbar_wait(&full[at.slot], at.parity, tmo, abort_flag) ||
                                                (it >= kAcc && !mbar_wait(&aempty[acc.slot], acc.parity ^ 1, tmo, abort_flag)))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t alo = base + at.slot * (bytes >> 4), blo = alo + (kWBytes >> 4);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    umma_e4m3_lead(lead, tm + acc.slot * kMostRows, alo + (kGrad ? 256 : 2) * i, blo + 2 * i, hi, idesc, i != 0);
                umma_commit_lead(lead, &empty[at.slot]);
                umma_commit_lead(lead, &afull[acc.slot]);
                __syncwarp();
            }
        }
        // every MMA is complete before TMEM and shared memory are released
        umma_commit_lead(lead, drain);
        if (__any_sync(0xffffffffu, !mbar_wait(drain, 0, tmo, nullptr))) ok = false;
    } else if (warp == 2) {
        // ------------------------------------------------------------ scales: lane = rows lane, lane + 32
        if (args.early) wait_for_prior_grid();
        const int wide = (args.cols + 127) / 128;
        const int64_t plane = static_cast<int64_t>(wide) * blocks, step = kGrad ? wide : 1;
        Place sc;
        int g = 0;
        for (int t = first; ok && t < count; t += stride) {
            const Tile x = tiles.at(t);
            const float *ws = args.weight_scales + x.e * plane + x.c0 / 128 * (kGrad ? 1 : static_cast<int64_t>(blocks)) + kb0 * step;
            const float *rs = args.row_scales + (static_cast<int64_t>(x.r0) + lane) * blocks + kb0;
            for (int b0 = 0; ok && b0 < own; b0 += 4) {
                float r[2][4], w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool in = b0 + j < own;
                    w[j] = in ? load_float(ws + (b0 + j) * step) : 0.f;
                    r[0][j] = in && lane < x.rows ? load_float(rs + b0 + j) : 0.f;
                    r[1][j] = in && lane + 32 < x.rows ? load_float(rs + 32 * static_cast<int64_t>(blocks) + b0 + j) : 0.f;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (b0 + j >= own) break;
                    if (g >= kScales && __any_sync(0xffffffffu, !mbar_wait(&sempty[sc.slot], sc.parity ^ 1, tmo, abort_flag))) {
                        ok = false;
                        break;
                    }
                    scales[sc.slot * kMostRows + lane] = r[0][j] * w[j];
                    scales[sc.slot * kMostRows + 32 + lane] = r[1][j] * w[j];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sfull[sc.slot]);
                    sc.next(kScales);
                    ++g;
                }
            }
        }
    } else if (warp == 3) {
        // ------------------------------------------------------------ rows of no expert
        if (args.early) wait_for_prior_grid();
        if (args.zero_rest) {
            zero_range(args.out, 0, static_cast<int64_t>(off[0]) * args.cols, lane);
            zero_range(args.out, static_cast<int64_t>(off[args.E]) * args.cols, static_cast<int64_t>(args.T) * args.cols, lane);
        }
    } else {
        // ------------------------------------------------------------ sums: lane = column of the output, column = row
        if (args.early) wait_for_prior_grid();
        const int q = warp & 3;
        const uint32_t mine = tmem + (static_cast<uint32_t>(32 * q) << 16);
        Place acc, sc;
        for (int t = first; ok && t < count; t += stride) {
            const Tile x = tiles.at(t);
            float y[kMostRows];
#pragma unroll
            for (int i = 0; i < kMostRows; ++i) y[i] = 0.f;
            for (int b = 0; b < own; ++b, acc.next(kAcc), sc.next(kScales)) {
                if (__any_sync(0xffffffffu, !mbar_wait(&sfull[sc.slot], sc.parity, tmo, abort_flag) ||
                                                !mbar_wait(&afull[acc.slot], acc.parity, tmo, abort_flag))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const float4 *s = reinterpret_cast<const float4 *>(scales + sc.slot * kMostRows);
#pragma unroll
                for (int j = 0; j < kMostRows / 16; ++j)
                    if (16 * j < x.n) {
                        uint32_t v[16];
                        tmem_ld16(mine + acc.slot * kMostRows + 16 * j, v);
                        float f[16];
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const float4 k = s[4 * j + u];
                            f[4 * u] = k.x, f[4 * u + 1] = k.y, f[4 * u + 2] = k.z, f[4 * u + 3] = k.w;
                        }
                        tmem_wait_ld();
#pragma unroll
                        for (int u = 0; u < 16; ++u) y[16 * j + u] = fmaf(__uint_as_float(v[u]), f[u], y[16 * j + u]);
                    }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&aempty[acc.slot]);
                    mbar_arrive(&sempty[sc.slot]);
                }
            }
            if (!ok) break;
            const int n = x.c0 + 32 * q + lane;
            if (parts > 1) {  // the only tile: all copies have landed and all MMAs are done, so the ring's place is free
                float *part = reinterpret_cast<float *>(stages);
#pragma unroll
                for (int r = 0; r < kMostRows; ++r)
                    if (r < x.rows) part[r * kPartStride + 32 * q + lane] = y[r];
            } else if (n < args.cols) {
                const float bias = args.bias ? __bfloat162float(args.bias[static_cast<int64_t>(x.e) * args.cols + n]) : 0.f;
                __nv_bfloat16 *out = args.out + static_cast<int64_t>(x.r0) * args.cols + n;
#pragma unroll
                for (int r = 0; r < kMostRows; ++r)
                    if (r < x.rows) out[r * static_cast<int64_t>(args.cols)] = __float2bfloat16(y[r] + bias);
            }
        }
    }
    __syncwarp();
    if (lane == 0 && !ok) {
        *abort_flag = 1;
        set_status(args.status, BSL_ERR_TIMEOUT);
    }
    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {  // a copy of a stage that was not armed ends by itself in some microseconds: wait a thousand
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000) __nanosleep(1000);
        __syncwarp();
    }
    if (parts > 1) {
        cluster_sync_all();
        if (first < count && !*abort_flag) {
            const Tile x = tiles.at(first);
            const float *part = reinterpret_cast<const float *>(stages);
            for (int i = rank * kThreads + threadIdx.x; i < x.rows * kCols; i += parts * kThreads) {
                const int r = i / kCols, f = i % kCols;
                float y = 0.f;
                for (int p = 0; p < parts; ++p) {
                    float other;
                    asm volatile("ld.shared::cluster.f32 %0, [%1];"
                                 : "=f"(other)
                                 : "r"(cluster_addr(part + r * kPartStride + f, p))
                                 : "memory");
                    y += other;
                }
                if (x.c0 + f >= args.cols) continue;
                if (args.bias) y += __bfloat162float(args.bias[static_cast<int64_t>(x.e) * args.cols + x.c0 + f]);
                args.out[(static_cast<int64_t>(x.r0) + r) * args.cols + x.c0 + f] = __float2bfloat16(y);
            }
        }
        cluster_sync_all();  // until the others have read this CTA's sums
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmem);
    }
}

}  // namespace

namespace {
int64_t most_tiles(int32_t T, int32_t E, int32_t cols)
{
    return static_cast<int64_t>((cols + kCols - 1) / kCols) * ((T < E ? T : E) + T / kMostRows);
}
}  // namespace

// Up to 64 rows an expert, on the average (us here / with fp8.cu: 384 rows in all on eight experts of 14336 x 4096
// 111 / 131, 512 118 / 129, 768 184 / 134), and more if that gives no more tiles than the SMs take at once, or
// little more (one of 4096 x 4096: 96 rows 22.5 / 28.7, 256 24.6 / 30.7; one of 11008 x 4096: 128 rows 38.9 / 30.7).
bool fp8_few(int32_t T, int32_t E, int32_t cols)
{
    return T <= static_cast<int64_t>(kMostRows) * E || (T <= 256ll * E && 4 * most_tiles(T, E, cols) <= 5 * num_sms());
}

bsl_status launch_fp8_few(const uint8_t *codes, const float *scales, int32_t T, const int32_t *offsets, const bsl_fp8 *W,
                          bool transposed, const void *bias, void *out, int32_t zero_rest, bool early, cudaStream_t s)
{
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
    args.early = early;
    args.timeout_ns = wait_timeout_ns();
    Maps m;
    const int64_t K = W->K, N = W->N;
    bool good = make_map_3d(&m.weight, W->codes, K / 2, N, W->E, K, K * N, 64, 128, 128);
    for (int i = 0; i < 4 && kStep * i < T; ++i)
        good = good && make_map_3d(&m.rows[i], codes, args.depth / 2, T, 1, args.depth, static_cast<uint64_t>(args.depth) * T, 64,
                                   kStep * (i + 1), 128);
    if (!good) return BSL_ERR_CUDA;
    auto kern = transposed ? k_fp8_few<true> : k_fp8_few<false>;
    const bsl_status sa = set_smem_once(reinterpret_cast<const void *>(kern), kSmem);
    if (sa != BSL_OK) return sa;
    // no more tiles than these; the clusters that cut the blocks have one each, and each CTA of theirs some blocks
    const int64_t tiles = most_tiles(T, W->E, args.cols);
    const int blocks = (args.depth + kBlock - 1) / kBlock;
    args.parts = 1;
    while (args.parts < 8 && 2 * args.parts * tiles <= num_sms() && 4 * args.parts <= blocks) args.parts *= 2;
    const int64_t grid = tiles * args.parts < num_sms() ? tiles * args.parts : num_sms();
    return cuda_status(launch_dependent_cluster(kern, static_cast<unsigned>(grid), args.parts, kThreads, kSmem, s, m, args));
}

}  // namespace bsl
