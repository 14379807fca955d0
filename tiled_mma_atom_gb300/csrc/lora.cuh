// lora.cuh — device pieces of the kernels of products with adapters: tile loads of
// rank 3, gathers, and MMAs that leave out rows (lanes) of the accumulator.
#pragma once

#include "device.cuh"

namespace tmg {

constexpr int kNoAdapter = 0x7fffffff;

__device__ __forceinline__ void tma_load_3d_one(void *dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1, int c2)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];\n\t}" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

// Counted on an mbarrier of the pair's CTA 0.
__device__ __forceinline__ void tma_load_3d_pair(void *dst, const CUtensorMap *map, uint32_t bar, int c0, int c1, int c2)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];\n\t}" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

// Four rows by number (out of range: zeros), issued by the calling lane.
__device__ __forceinline__ void tma_gather4_one(void *dst, const CUtensorMap *map, uint64_t *bar, int c0, const int4 &r)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(dst)),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w)
                 : "memory");
}

// One MMA of the CTA, and one of the pair, that updates the rows (lanes) whose bit in
// `off` is clear.
__device__ __forceinline__ void mma_bf16_masked_w(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                  const uint4 &off, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %8, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, {%4, %5, %6, %7}, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(off.x), "r"(off.y), "r"(off.z), "r"(off.w), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void mma_bf16_pair_masked_w(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                       const uint32_t (&off)[8])
{
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.eq.b32 p, 0, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, {%4, %5, %6, %7, %8, %9, %10, %11}, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(off[0]), "r"(off[1]), "r"(off[2]), "r"(off[3]), "r"(off[4]), "r"(off[5]),
        "r"(off[6]), "r"(off[7])
        : "memory");
}

// Eight consecutive floats at the same shared-memory place in the S <= 8 CTAs of the
// cluster, summed in rank order; all loads in flight together.
__device__ __forceinline__ void cluster_sum8(uint32_t at, uint32_t S, float (&z)[8])
{
    float4 a[8], b[8];
#pragma unroll
    for (uint32_t s = 0; s < 8; ++s)
        if (s < S) {
            const uint32_t there = mapa_shared(at, s);
            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(a[s].x), "=f"(a[s].y), "=f"(a[s].z), "=f"(a[s].w) : "r"(there));
            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(b[s].x), "=f"(b[s].y), "=f"(b[s].z), "=f"(b[s].w) : "r"(there + 16));
        }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        z[i] = 0.f;
#pragma unroll
    for (uint32_t s = 0; s < 8; ++s)
        if (s < S) {
            z[0] += a[s].x, z[1] += a[s].y, z[2] += a[s].z, z[3] += a[s].w;
            z[4] += b[s].x, z[5] += b[s].y, z[6] += b[s].z, z[7] += b[s].w;
        }
}

// The adapters of 32 W rows from row0 on: lane i has those of rows 32 w + i, kNoAdapter
// where there is none (rows past M, numbers outside 0 .. L - 1).  Read past L1: before
// the kernel's own wait.
template <int W>
struct RowAdapters {
    int id[W];

    __device__ __forceinline__ void read(const int32_t *adapters, int64_t row0, int64_t M, int L, int lane)
    {
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const int64_t m = row0 + 32 * w + lane;
            const int l = m < M ? __ldcg(adapters + m) : -1;
            id[w] = l >= 0 && l < L ? l : kNoAdapter;
        }
    }
    // The smallest above `last`; kNoAdapter after the largest.
    __device__ __forceinline__ int next(int last) const
    {
        int least = kNoAdapter;
#pragma unroll
        for (int w = 0; w < W; ++w)
            least = id[w] > last ? min(least, id[w]) : least;
        return __reduce_min_sync(0xffffffffu, least);
    }
    // The rows that adapter l leaves out.
    __device__ __forceinline__ void others(int l, uint32_t (&off)[W]) const
    {
#pragma unroll
        for (int w = 0; w < W; ++w)
            off[w] = ~__ballot_sync(0xffffffffu, id[w] == l);
    }
};

}  // namespace tmg
