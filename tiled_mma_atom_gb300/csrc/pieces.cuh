// pieces.cuh — tiles whose contraction is split between CTA pairs: each pair
// leaves fp32 partial sums in workspace, the last to arrive adds them up in
// pair order, so the result does not depend on timing.
#pragma once

#include "device.cuh"

namespace tmg {

// A warp has stored its piece of a split tile: arrive on the tile's counter;
// true for the last of `others` + 1 arrivals, which then sees every piece.  The
// warp's stores come before lane 0's release by the first syncwarp, its lanes' reads
// of the pieces after lane 0's acquire by the second (a shuffle orders no memory).
__device__ __forceinline__ bool last_arrival(uint32_t *counter, int others, bool ok)
{
    uint32_t old = 0;
    __syncwarp();
    if ((threadIdx.x & 31) == 0 && ok) {
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(old) : "l"(counter) : "memory");
        if (old == static_cast<uint32_t>(others))
            *counter = 0;
    }
    __syncwarp();
    return __shfl_sync(0xffffffffu, old, 0) == static_cast<uint32_t>(others) && others >= 0;
}

// v += the pieces of pairs c0 .. c1 in that order (base(cc): a pair's piece,
// `in`: this thread's place in its chunk), two pieces' loads in flight.
template <class Base>
__device__ __forceinline__ void add_pieces(float (&v)[32], const float *partials, int64_t limit, int64_t in, int c0, int c1,
                                           Base &&base, const ErrCtx &err)
{
    for (int cc = c0; cc <= c1; cc += 2) {
        float4 f[2][8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t at = cc + i <= c1 ? base(cc + i) + in : 0;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                f[i][j] = cc + i <= c1 && span_ok(at + j * 128, 4, limit, err, kBndPartials)
                              ? __ldcg(reinterpret_cast<const float4 *>(partials + at + j * 128))
                              : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[4 * j] += f[i][j].x;
                v[4 * j + 1] += f[i][j].y;
                v[4 * j + 2] += f[i][j].z;
                v[4 * j + 3] += f[i][j].w;
            }
    }
}

}  // namespace tmg
