// copy.cuh — operand rows that TMA boxes do not cover (the end of a group)
// copied into the ring by warps: 16-byte cp.async, zero-filled where there is
// no source, handed to the MMA issuer of the pair.
//
// cp.async writes through the generic proxy and the MMA reads through the
// async proxy, possibly from the other CTA: a warp waits for its own copies,
// each lane fences its writes, and one lane arrives on CTA 0's `full` barrier
// with a release at cluster scope.  That release takes about 1.1 us of the
// warp, so it is for a group's last block; blocks without copies arrive with
// the CTA-scope release, which has nothing to hand over.
#pragma once

#include "device.cuh"

namespace tmg {

constexpr int kCopyWarps = 4;

// `bytes` (0..16) of src, the rest of the 16 bytes zero; both 16-byte aligned.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// This thread's copies have landed and are ordered before async-proxy reads.
__device__ __forceinline__ void copies_done()
{
    asm volatile("cp.async.wait_all;\n\tfence.proxy.async.shared::cta;" ::: "memory");
}

// Whole warp, after copies_done(): one arrival on CTA 0's barrier.
__device__ __forceinline__ void arrive_copied(uint64_t *bar)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(mapa_shared(smem_u32(bar), 0))
                     : "memory");
}

}  // namespace tmg
