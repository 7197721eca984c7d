// ring.cuh -- weight rows streamed to few tokens: rings of asynchronous copies that
// feed mma.sync (moe.cu's two kernels).
//
// A step is 128 bytes of 16 weight rows.  A warp brings its steps through a ring of
// its own in shared memory, by copies that need no registers, Ring of them under way
// whatever is summed meanwhile, over the borders of units of work too.  In a step's
// rows the 16-byte units of odd rows trade halves, so that a lane's reads (units t and
// 4 + t of rows g and g + 8, the MMA's A operand; k in the order in which the bytes
// lie) meet no bank twice.
//
// The warps of a CTA work in teams that cut a unit's steps: all eight where there are
// steps enough, else fewer, so that a warp has some steps for each time the team adds
// up its sums.
#pragma once

#include "common.cuh"

namespace bsl {

constexpr int kWarps = 8;
constexpr int kStep = 16 * 128;
constexpr int kRows = 8;  // tokens in a group (MMA N)

// Four copies a lane: unit lane & 7 of rows lane / 8 + 4 j at `from` + off[j]; zeros where there is none.
__device__ __forceinline__ void copy_step(uint8_t *slot, const uint8_t *from, const int64_t (&off)[4], const bool (&exists)[4],
                                          const uint8_t *any)
{
    const int lane = threadIdx.x & 31, r = lane >> 3, u = lane & 7;
    const uint32_t dst = smem_u32(slot) + r * 128 + ((u ^ (r & 1) << 2) << 4);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + j * 512), "l"(exists[j] ? from + off[j] : any),
                     "r"(exists[j] ? 16 : 0)
                     : "memory");
}

__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// The oldest step of Ring is there, for the whole warp.
template <int Ring>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(Ring - 1) : "memory");
    __syncwarp();
}

__device__ __forceinline__ void copies_end() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// A lane's 16 bytes of row g (and of row g + 8) in half h of a step.
__device__ __forceinline__ void read_step(const uint8_t *slot, int h, uint4 &lo, uint4 &hi)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint8_t *at = slot + g * 128 + (((4 * h + t) ^ (g & 1) << 2) << 4);
    lo = *reinterpret_cast<const uint4 *>(at);
    hi = *reinterpret_cast<const uint4 *>(at + 1024);
}

// Warps of a team for units of so many steps.
inline int team_of(int steps) { return steps >= 4 * kWarps ? kWarps : steps >= 2 * kWarps ? kWarps / 2 : kWarps / 4; }

}  // namespace bsl
