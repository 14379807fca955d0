// route.cuh — the choice of a token's experts, for the kernels that route: route.cu
// says how.
#pragma once

#include <cuda_bf16.h>

#include "grouped.h"

namespace tmg {
namespace {

constexpr uint32_t kFull = 0xffffffffu;

constexpr float kNegInf = -__builtin_huge_valf();

__device__ __forceinline__ float load_logit(const void *p, int64_t i, bool bf16)
{
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]) : static_cast<const float *>(p)[i];
}

// The same past L1, for a kernel that reads them before its own wait (launch.cuh).
__device__ __forceinline__ float load_logit_l2(const void *p, int64_t i, bool bf16)
{
    if (!bf16)
        return __ldcg(static_cast<const float *>(p) + i);
    const unsigned short w = __ldcg(static_cast<const unsigned short *>(p) + i);
    return __uint_as_float(static_cast<uint32_t>(w) << 16);
}

// Key of a logit: 0 for -inf and NaN, else increasing with the value (adding
// +0 makes the two zeros equal).
__device__ __forceinline__ uint32_t logit_key(float x)
{
    if (!(x > kNegInf))
        return 0;
    const uint32_t u = __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float key_logit(uint32_t key)
{
    return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// e^(x - top), 1 where x is the largest itself (also at +inf).
__device__ __forceinline__ float exp_from(float x, float top) { return x == top ? 1.f : expf(x - top); }

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(kFull, v, o);
    return v;
}

// The choices of tokens t0 .. t1 - 1, one warp per token; counts (shared) gets
// each expert's number; pairs (shared, or null) the chosen experts in order.
template <int C, bool BF16, bool L2 = false>
__device__ __forceinline__ void choose(const RouteArgs &a, int64_t t0, int64_t t1, int32_t *counts, int32_t *pairs)
{
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    float next[C];               // the warp's next token's logits, in flight
    auto fetch = [&](int64_t t) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = lane + 32 * c;
            next[c] = t >= t1 || e >= a.E ? kNegInf
                      : L2                ? load_logit_l2(a.logits, t * a.ld + e, BF16)
                                          : load_logit(a.logits, t * a.ld + e, BF16);
        }
    };
    fetch(t0 + warp);
    for (int64_t t = t0 + warp; t < t1; t += warps) {
        uint32_t key[C];
#pragma unroll
        for (int c = 0; c < C; ++c)
            key[c] = logit_key(next[c]);
        fetch(t + warps);
        float sum_all = 0.f;
        if (!a.normalize) {
            uint32_t all = 0;
#pragma unroll
            for (int c = 0; c < C; ++c)
                all = max(all, key[c]);
            all = __reduce_max_sync(kFull, all);
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (key[c])
                    sum_all += exp_from(key_logit(key[c]), key_logit(all));
            sum_all = warp_sum(sum_all);
        }
        if constexpr (BF16) {
            // a bf16's fp32 key ends in sixteen equal bits: zeros above, ones
            // below zero
#pragma unroll
            for (int c = 0; c < C; ++c)
                key[c] = key[c] ? (key[c] & 0xffff0000u) | (0xffffu - static_cast<uint32_t>(lane + 32 * c)) : 0;
        }
        uint32_t mine_key = 0;       // lane j < k: the j-th choice
        int mine = -1;
        for (int j = 0; j < a.k; ++j) {
            uint32_t best = 0, top;
            int e;
            if constexpr (BF16) {
#pragma unroll
                for (int c = 0; c < C; ++c)
                    best = max(best, key[c]);
                top = __reduce_max_sync(kFull, best);
                if (top == 0)
                    break;
                e = static_cast<int>(0xffffu - (top & 0xffffu));
#pragma unroll
                for (int c = 0; c < C; ++c)
                    if (key[c] == top)
                        key[c] = 0;
                top = top & 0x80000000u ? top & 0xffff0000u : top | 0xffffu;
            } else {
                int at = 0x7fffffff;
#pragma unroll
                for (int c = 0; c < C; ++c)
                    if (key[c] > best) {
                        best = key[c];
                        at = lane + 32 * c;
                    }
                top = __reduce_max_sync(kFull, best);
                if (top == 0)
                    break;
                e = static_cast<int>(__reduce_min_sync(kFull, best == top ? static_cast<uint32_t>(at) : 0x7fffffffu));
#pragma unroll
                for (int c = 0; c < C; ++c)
                    if (lane + 32 * c == e)
                        key[c] = 0;
            }
            if (lane == j) {
                mine_key = top;
                mine = e;
            }
        }
        const float top = key_logit(__shfl_sync(kFull, mine_key, 0));
        const float ex = mine >= 0 ? exp_from(key_logit(mine_key), top) : 0.f;
        const float sum = a.normalize ? warp_sum(ex) : sum_all;
        if (lane < a.k) {
            a.weights[t * a.k + lane] = mine >= 0 ? ex / sum : 0.f;
            a.experts[t * a.k + lane] = mine;
            if (pairs)
                pairs[(t - t0) * a.k + lane] = mine;
            if (mine >= 0)
                atomicAdd(&counts[mine], 1);
        }
    }
}

}  // namespace
}  // namespace tmg
