// staging.cuh — 16-byte pieces between registers, shared memory and the rows of
// an output matrix.
#pragma once

#include <cuda_bf16.h>

#include "device.cuh"

namespace tmg {

__device__ __forceinline__ uint4 lds128(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void sts128(uint32_t addr, const uint4 &v)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Eight bf16 of an output row at element offset `off`, `n` (1..8) of them inside
// the row: one 16-byte store where all are and the address allows it.
__device__ __forceinline__ void store_piece(__nv_bfloat16 *M, int64_t off, const uint4 &v, int n, int64_t limit,
                                            const ErrCtx &err)
{
    if (!span_ok(off, n, limit, err, kBndStoreD))
        return;
    __nv_bfloat16 *p = M + off;
    if (n == 8 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
        *reinterpret_cast<uint4 *>(p) = v;
    } else {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n)
                reinterpret_cast<uint16_t *>(p)[j] = static_cast<uint16_t>(w[j / 2] >> (16 * (j & 1)));
    }
}

}  // namespace tmg
