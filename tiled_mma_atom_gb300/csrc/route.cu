// route.cu — routing of tokens to experts: the k largest logits of each
// token, their weights, and the plan that sorts the (token, choice) pairs by
// expert for the grouped products; the weights' gradient; and the weighted
// sum of the experts' answers with its gradient.
//
// Selection.  One warp per token, expert e = lane + 32 c in register c.
// Logits map to unsigned keys of the same order (sign bit flipped, negative
// values inverted); -inf and NaN map to 0, which is never selected.  Each of
// the k steps is a warp-wide maximum of the keys and a warp-wide minimum of
// the experts that hold it (two redux instructions), so equal logits go to
// the lowest expert.
//
// Plan.  A stable counting sort.  Blocks take contiguous runs of tokens and
// leave their counts per expert; the second kernel adds up the counts of
// experts and blocks before its own and ranks its pairs in order: 32 pairs at
// a time per warp, the lanes with the same expert found by match.any.  No
// atomic decides an order, so the plan does not depend on timing.
#include <cuda_bf16.h>

#include <algorithm>

#include "grouped.h"

namespace tmg {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr float kNegInf = -__builtin_huge_valf();

__device__ __forceinline__ float load_logit(const void *p, int64_t i, bool bf16)
{
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]) : static_cast<const float *>(p)[i];
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

template <int C>
__global__ void __launch_bounds__(256) route_topk_kernel(RouteArgs a, int tokens_per_block)
{
    extern __shared__ int32_t counts[];
    for (int e = threadIdx.x; e < a.E; e += blockDim.x)
        counts[e] = 0;
    __syncthreads();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tokens_per_block;
    const int64_t t1 = min(a.T, t0 + tokens_per_block);
    for (int64_t t = t0 + warp; t < t1; t += warps) {
        uint32_t key[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = lane + 32 * c;
            key[c] = e < a.E ? logit_key(load_logit(a.logits, t * a.ld + e, a.bf16)) : 0;
        }
        uint32_t all = 0;
        float sum_all = 0.f;
        if (!a.normalize) {
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
        uint32_t mine_key = 0;       // lane j < k: the j-th choice
        int mine = -1;
        for (int j = 0; j < a.k; ++j) {
            uint32_t best = 0;
            int at = 0x7fffffff;
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (key[c] > best) {
                    best = key[c];
                    at = lane + 32 * c;
                }
            const uint32_t top = __reduce_max_sync(kFull, best);
            if (top == 0)
                break;
            const int e = static_cast<int>(__reduce_min_sync(kFull, best == top ? static_cast<uint32_t>(at) : 0x7fffffffu));
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (lane + 32 * c == e)
                    key[c] = 0;
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
            if (mine >= 0)
                atomicAdd(&counts[mine], 1);
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += blockDim.x)
        a.counts[static_cast<int64_t>(blockIdx.x) * a.E + e] = counts[e];
}

// Shared memory: base[E], warp counts [warps][E], scan scratch [33].
__global__ void __launch_bounds__(256) route_plan_kernel(RouteArgs a, int tokens_per_block, int blocks)
{
    extern __shared__ int32_t sm[];
    const int E = a.E, warps = blockDim.x / 32, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int32_t *base = sm, *wc = sm + E, *total = wc + warps * E;
    // counts of this expert in the blocks before, and in all of them
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        int before = 0, sum = 0;
        for (int b = 0; b < blocks; ++b) {
            const int n = __ldg(a.counts + static_cast<int64_t>(b) * E + e);
            if (b < static_cast<int>(blockIdx.x))
                before += n;
            sum += n;
        }
        base[e] = before;
        total[e] = sum;
    }
    for (int i = threadIdx.x; i < warps * E; i += blockDim.x)
        wc[i] = 0;
    __syncthreads();
    if (warp == 0) {                 // exclusive prefix over the experts
        int run = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane, n = e < E ? total[e] : 0;
            int inc = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(kFull, inc, o);
                if (lane >= o)
                    inc += v;
            }
            if (e < E) {
                base[e] += run + inc - n;
                if (blockIdx.x == 0)
                    a.offsets[e] = run + inc - n;
            }
            run += __shfl_sync(kFull, inc, 31);
        }
        if (lane == 0) {
            total[0] = run;
            if (blockIdx.x == 0)
                a.offsets[E] = run;
        }
    }
    const int64_t p0 = static_cast<int64_t>(blockIdx.x) * tokens_per_block * a.k;
    const int64_t p1 = min(a.T * a.k, p0 + static_cast<int64_t>(tokens_per_block) * a.k);
    // each warp's pairs are contiguous: [w0, w1)
    const int64_t each = ((p1 - p0 + warps - 1) / warps + 31) / 32 * 32;
    const int64_t w0 = min(p1, p0 + warp * each), w1 = min(p1, w0 + each);
    for (int64_t p = w0; p < w1; p += 32) {
        const int e = p + lane < w1 ? a.experts[p + lane] : -1;
        const uint32_t same = __match_any_sync(kFull, e);
        if (e >= 0 && lane == __ffs(same) - 1)
            wc[warp * E + e] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    const int rows_used = total[0];
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        int run = base[e];
        for (int w = 0; w < warps; ++w) {
            const int n = wc[w * E + e];
            wc[w * E + e] = run;
            run += n;
        }
    }
    __syncthreads();
    for (int64_t p = w0; p < w1; p += 32) {
        const int64_t i = p + lane;
        const int e = i < w1 ? a.experts[i] : -1;
        const uint32_t same = __match_any_sync(kFull, e);
        const int first = e >= 0 ? wc[warp * E + e] : 0;
        __syncwarp();
        if (e >= 0) {
            const int slot = first + __popc(same & ((1u << lane) - 1));
            if (lane == __ffs(same) - 1)
                wc[warp * E + e] = first + __popc(same);
            a.slots[i] = slot;
            a.rows[slot] = static_cast<int32_t>(i / a.k);
        } else if (i < w1) {
            a.slots[i] = -1;
        }
        __syncwarp();
    }
    // rows that no pair takes
    for (int64_t i = rows_used + static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < a.T * a.k;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x)
        a.rows[i] = -1;
}

// Gradient of the weights.  With the softmax over the selected logits,
// dlogit_j = w_j (dw_j - sum_i w_i dw_i) at the selected ones and 0 elsewhere;
// with the softmax p over all, dlogit_e = p_e ([e selected] dw - sum_i p_i dw_i).
template <int C>
__global__ void __launch_bounds__(256)
    route_backward_kernel(const void *__restrict__ logits, bool bf16, int64_t T, int64_t ld, int E, int k, bool normalize,
                          const int32_t *__restrict__ experts, const float *__restrict__ dweights, void *__restrict__ out)
{
    const int lane = threadIdx.x % 32;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x / 32);
    for (int64_t t = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) / 32; t < T; t += warps) {
        int e = -1;
        float dw = 0.f, x = kNegInf;
        if (lane < k) {
            e = experts[t * k + lane];
            if (e < 0 || e >= E)
                e = -1;
            else {
                dw = dweights[t * k + lane];
                x = load_logit(logits, t * ld + e, bf16);
            }
        }
        const float top = __shfl_sync(kFull, x, 0);       // the first choice is the largest
        float ex = e >= 0 ? exp_from(x, top) : 0.f;
        float v[C], sum = 0.f;
        if (normalize) {
            sum = ex;
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int i = lane + 32 * c;
                const float l = i < E ? load_logit(logits, t * ld + i, bf16) : kNegInf;
                v[c] = l > kNegInf ? exp_from(l, top) : 0.f;
                sum += v[c];
            }
        }
        sum = warp_sum(sum);
        const float w = e >= 0 ? ex / sum : 0.f;
        const float mean = warp_sum(w * dw);
        const float g = w * (dw - (normalize ? mean : 0.f));
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = lane + 32 * c;
            float d = !normalize && v[c] != 0.f ? -(v[c] / sum) * mean : 0.f;
            for (int j = 0; j < k; ++j) {
                const int ej = __shfl_sync(kFull, e, j);
                const float gj = __shfl_sync(kFull, g, j);
                if (ej == i)
                    d += gj;
            }
            if (i < E) {
                if (bf16)
                    static_cast<__nv_bfloat16 *>(out)[t * E + i] = __float2bfloat16_rn(d);
                else
                    static_cast<float *>(out)[t * E + i] = d;
            }
        }
    }
}

// ------------------------------------------------------------- combine

__device__ __forceinline__ void unpack8(const uint4 &w, float (&f)[8])
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(u[i] << 16);
        f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// Eight columns from h (fewer at the end of the row) of a bf16 row.
template <bool VEC>
__device__ __forceinline__ void load8(const __nv_bfloat16 *row, int64_t h, int64_t H, float (&f)[8])
{
    if constexpr (VEC) {
        unpack8(*reinterpret_cast<const uint4 *>(row + h), f);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = h + i < H ? __bfloat162float(row[h + i]) : 0.f;
    }
}

template <bool VEC>
__device__ __forceinline__ void store8(__nv_bfloat16 *row, int64_t h, int64_t H, const float (&f)[8])
{
    if constexpr (VEC) {
        *reinterpret_cast<uint4 *>(row + h) = pack8(f);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (h + i < H)
                row[h + i] = __float2bfloat16_rn(f[i]);
    }
}

constexpr int kCombineThreads = 128;

template <bool VEC>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(CombineArgs a, int64_t parts)
{
    const int64_t t = blockIdx.x / parts;
    const int64_t h = ((blockIdx.x % parts) * kCombineThreads + threadIdx.x) * 8;
    if (h >= a.H)
        return;
    float acc[8] = {};
    if (a.residual)
        load8<VEC>(static_cast<const __nv_bfloat16 *>(a.residual) + t * a.ldr, h, a.H, acc);
    const __nv_bfloat16 *Y = static_cast<const __nv_bfloat16 *>(a.Y);
    for (int j = 0; j < a.k; ++j) {
        const int64_t slot = __ldg(a.slots + t * a.k + j);
        if (slot < 0 || slot >= a.R)
            continue;
        const float w = a.weights ? __ldg(a.weights + t * a.k + j) : 1.f;
        float y[8];
        load8<VEC>(Y + slot * a.ldy, h, a.H, y);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            acc[i] = fmaf(w, y[i], acc[i]);
    }
    store8<VEC>(static_cast<__nv_bfloat16 *>(a.out) + t * a.ldo, h, a.H, acc);
}

constexpr int kMaxChoices = 16;

template <bool VEC>
__global__ void __launch_bounds__(256) combine_backward_kernel(CombineGradArgs a)
{
    __shared__ float part[8][kMaxChoices];
    const int64_t t = blockIdx.x;
    float dot[kMaxChoices];
#pragma unroll
    for (int j = 0; j < kMaxChoices; ++j)
        dot[j] = 0.f;
    for (int64_t h = threadIdx.x * 8; h < a.H; h += 256 * 8) {
        float d[8];
        load8<VEC>(static_cast<const __nv_bfloat16 *>(a.dOut) + t * a.ldo, h, a.H, d);
#pragma unroll
        for (int j = 0; j < kMaxChoices; ++j) {
            if (j >= a.k)
                break;
            const int64_t slot = __ldg(a.slots + t * a.k + j);
            if (slot < 0 || slot >= a.R)
                continue;
            const float w = a.weights ? __ldg(a.weights + t * a.k + j) : 1.f;
            if (a.dweights) {
                float y[8];
                load8<VEC>(static_cast<const __nv_bfloat16 *>(a.Y) + slot * a.ldy, h, a.H, y);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    dot[j] = fmaf(d[i], y[i], dot[j]);
            }
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                o[i] = w * d[i];
            store8<VEC>(static_cast<__nv_bfloat16 *>(a.dY) + slot * a.H, h, a.H, o);
        }
    }
    if (!a.dweights)
        return;
#pragma unroll
    for (int j = 0; j < kMaxChoices; ++j) {
        if (j >= a.k)
            break;
        const float v = warp_sum(dot[j]);
        if (threadIdx.x % 32 == 0)
            part[threadIdx.x / 32][j] = v;
    }
    __syncthreads();
    if (threadIdx.x < a.k) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w)
            v += part[w][threadIdx.x];
        a.dweights[t * a.k + threadIdx.x] = v;
    }
}

int tokens_per_block(int64_t T, int num_sms) { return static_cast<int>((T + num_sms - 1) / num_sms); }

bool vec8(const void *p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 8 == 0; }

}  // namespace

int route_blocks(int64_t T, int num_sms)
{
    const int each = tokens_per_block(T, num_sms);
    return static_cast<int>((T + each - 1) / each);
}

cudaError_t launch_route(const RouteArgs &a, int num_sms, cudaStream_t s)
{
    const int each = tokens_per_block(a.T, num_sms), blocks = route_blocks(a.T, num_sms);
    const size_t sm1 = a.E * sizeof(int32_t), sm2 = (10 * static_cast<size_t>(a.E)) * sizeof(int32_t);
    note_launch();
    if (a.E <= 64)
        route_topk_kernel<2><<<blocks, 256, sm1, s>>>(a, each);
    else if (a.E <= 256)
        route_topk_kernel<8><<<blocks, 256, sm1, s>>>(a, each);
    else
        route_topk_kernel<32><<<blocks, 256, sm1, s>>>(a, each);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    note_launch();
    route_plan_kernel<<<blocks, 256, sm2, s>>>(a, each, blocks);
    return cudaGetLastError();
}

cudaError_t launch_route_backward(const void *logits, bool bf16, int64_t T, int64_t ld, int E, int k, bool normalize,
                                  const int32_t *experts, const float *dweights, void *dlogits, int num_sms,
                                  cudaStream_t s)
{
    const int blocks = static_cast<int>(std::min<int64_t>((T + 7) / 8, num_sms * 8));
    note_launch();
    if (E <= 64)
        route_backward_kernel<2><<<blocks, 256, 0, s>>>(logits, bf16, T, ld, E, k, normalize, experts, dweights, dlogits);
    else if (E <= 256)
        route_backward_kernel<8><<<blocks, 256, 0, s>>>(logits, bf16, T, ld, E, k, normalize, experts, dweights, dlogits);
    else
        route_backward_kernel<32><<<blocks, 256, 0, s>>>(logits, bf16, T, ld, E, k, normalize, experts, dweights, dlogits);
    return cudaGetLastError();
}

cudaError_t launch_combine(const CombineArgs &a, cudaStream_t s)
{
    const int64_t parts = (a.H + kCombineThreads * 8 - 1) / (kCombineThreads * 8);
    const bool vec = a.H % 8 == 0 && vec8(a.Y, a.ldy) && vec8(a.out, a.ldo) && (!a.residual || vec8(a.residual, a.ldr));
    note_launch();
    if (vec)
        combine_kernel<true><<<static_cast<unsigned>(a.T * parts), kCombineThreads, 0, s>>>(a, parts);
    else
        combine_kernel<false><<<static_cast<unsigned>(a.T * parts), kCombineThreads, 0, s>>>(a, parts);
    return cudaGetLastError();
}

cudaError_t launch_combine_backward(const CombineGradArgs &a, cudaStream_t s)
{
    const bool vec = a.H % 8 == 0 && vec8(a.Y, a.ldy) && vec8(a.dOut, a.ldo) && vec8(a.dY, a.H);
    note_launch();
    if (vec)
        combine_backward_kernel<true><<<static_cast<unsigned>(a.T), 256, 0, s>>>(a);
    else
        combine_backward_kernel<false><<<static_cast<unsigned>(a.T), 256, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace tmg
