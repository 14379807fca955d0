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
// the lowest expert.  A bf16 logit's key has 16 bits: with the inverted expert
// number below it, one maximum finds both.
//
// Plan.  A stable counting sort.  Blocks take contiguous runs of tokens and
// leave their counts per expert (16 bits); a block of the second kernel takes
// two such runs, adds up the counts of experts and runs before its own and
// ranks its pairs in order: 32 pairs at a time per warp, the lanes with the
// same expert found by match.any.  Atomics
// only count, none decides an order, so the plan does not depend on timing.
// Up to kOneBlockTokens tokens one block does it all in one launch: beyond,
// its warps' tokens in a row cost more than the second launch.
#include <cuda_bf16.h>

#include <algorithm>

#include "grouped.h"
#include "launch.cuh"
#include "route.cuh"

namespace tmg {
namespace {

// Entries of a row of the counts table (8-byte rows of 16-bit counts).
__host__ __device__ __forceinline__ int count_row(int E) { return (E + 3) & ~3; }

// Warp 0: base[e] += the pairs of all experts before e; block 0 writes the
// offsets.  Returns the number of all pairs (in warp 0).
__device__ __forceinline__ int add_expert_prefix(const RouteArgs &a, int32_t *base, const int32_t *total)
{
    const int lane = threadIdx.x % 32;
    int run = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
        const int e = e0 + lane, n = e < a.E ? total[e] : 0;
        int inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kFull, inc, o);
            if (lane >= o)
                inc += v;
        }
        if (e < a.E) {
            base[e] += run + inc - n;
            if (blockIdx.x == 0)
                a.offsets[e] = run + inc - n;
        }
        run += __shfl_sync(kFull, inc, 31);
    }
    if (lane == 0 && blockIdx.x == 0)
        a.offsets[a.E] = run;
    return run;
}

// Slots and rows of the pairs p0 .. p1 - 1, whose experts are pairs[p - p0];
// base[e]: the first slot of this block's pairs of expert e.  wc: warps x E
// counters, zero.
__device__ __forceinline__ void rank_pairs(const RouteArgs &a, int p0, int p1, const int32_t *pairs, const int32_t *base,
                                           int32_t *wc)
{
    const int E = a.E, lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    const unsigned k = a.k;
    // each warp's pairs are contiguous: p0 + [w0, w1), with room for what lies past
    // the last pair (p0 itself may be near 2^31)
    const int here = p1 - p0, each = ((here + 31) / 32 + warps - 1) / warps * 32;
    const int w0 = min(here, warp * each), w1 = min(here, w0 + each);
    int32_t *mine = wc + warp * E;
    for (int p = w0; p < w1; p += 32) {
        const int e = p + lane < w1 ? pairs[p + lane] : -1;
        const uint32_t same = __match_any_sync(kFull, e);
        if (e >= 0 && lane == __ffs(same) - 1)
            mine[e] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        int run = base[e];
        for (int w = 0; w < warps; w += 8) {
            int n[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                n[i] = w + i < warps ? wc[(w + i) * E + e] : 0;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (w + i < warps) {
                    wc[(w + i) * E + e] = run;
                    run += n[i];
                }
        }
    }
    __syncthreads();
    for (int p = w0; p < w1; p += 32) {
        const int i = p + lane;
        const int e = i < w1 ? pairs[i] : -1;
        const uint32_t same = __match_any_sync(kFull, e);
        const int first = e >= 0 ? mine[e] : 0;
        __syncwarp();
        if (e >= 0) {
            const int slot = first + __popc(same & ((1u << lane) - 1));
            if (lane == __ffs(same) - 1)
                mine[e] = first + __popc(same);
            a.slots[p0 + i] = slot;
            a.rows[slot] = static_cast<int>(static_cast<unsigned>(p0 + i) / k);
        } else if (i < w1) {
            a.slots[p0 + i] = -1;
        }
        __syncwarp();
    }
}

// One block.  Shared memory: counts (totals) [E], base [E], pairs [T k], warp
// counters [warps][E].
template <int C, bool BF16>
__global__ void __launch_bounds__(1024) route_one_kernel(RouteArgs a)
{
    extern __shared__ int32_t sm[];
    __shared__ int used;
    const int warps = blockDim.x / 32;
    int32_t *counts = sm, *base = sm + a.E, *wc = base + a.E, *pairs = wc + warps * a.E;
    for (int i = threadIdx.x; i < (2 + warps) * a.E; i += blockDim.x)
        sm[i] = 0;
    grid_release();
    grid_wait();
    __syncthreads();
    choose<C, BF16>(a, 0, a.T, counts, pairs);
    __syncthreads();
    if (threadIdx.x < 32) {
        const int n = add_expert_prefix(a, base, counts);
        if (threadIdx.x == 0)
            used = n;
    }
    __syncthreads();
    const int all = static_cast<int>(a.T) * a.k;
    rank_pairs(a, 0, all, pairs, base, wc);
    for (int i = used + threadIdx.x; i < all; i += blockDim.x)
        a.rows[i] = -1;              // rows that no pair takes
}

template <int C, bool BF16>
__global__ void __launch_bounds__(1024) route_choose_kernel(RouteArgs a, int tokens_per_block)
{
    extern __shared__ int32_t counts[];
    for (int e = threadIdx.x; e < a.E; e += blockDim.x)
        counts[e] = 0;
    grid_release();
    grid_wait();
    __syncthreads();
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tokens_per_block;
    choose<C, BF16>(a, t0, min(a.T, t0 + tokens_per_block), counts, nullptr);
    __syncthreads();
    const int row = count_row(a.E);
    for (int e = threadIdx.x; e < row; e += blockDim.x)
        a.counts[static_cast<int64_t>(blockIdx.x) * row + e] = e < a.E ? static_cast<uint16_t>(counts[e]) : 0;
}

// Shared memory: base [E], totals [E], warp counters [warps][E], the block's
// pairs where they fit (kPlanPairs).
constexpr int kPlanPairs = 4096;
__global__ void __launch_bounds__(1024) route_plan_kernel(RouteArgs a, int tokens_per_block, int runs)
{
    extern __shared__ int32_t sm[];
    __shared__ int used;
    const int E = a.E, warps = blockDim.x / 32, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int32_t *base = sm, *total = sm + E, *wc = total + E;
    for (int i = threadIdx.x; i < (2 + warps) * E; i += blockDim.x)
        sm[i] = 0;
    grid_release();
    grid_wait();
    // this block's pairs, in flight together with the counts
    const int all = static_cast<int>(a.T * a.k), span = 2 * tokens_per_block * a.k;
    const int p0 = blockIdx.x * span, p1 = all - p0 < span ? all : p0 + span;
    const int32_t *pairs = a.experts + p0;
    if (span <= kPlanPairs) {
        int32_t *here = wc + warps * E;
        for (int i = threadIdx.x; i < p1 - p0; i += blockDim.x)
            here[i] = pairs[i];
        pairs = here;
    }
    __syncthreads();
    // counts in the runs before this block's, and in all: each warp adds up
    // every warps-th run, 128 experts at a time, four per lane
    const int row = count_row(E), first = 2 * blockIdx.x;
    for (int e0 = 0; e0 < E; e0 += 128) {
        int before[4] = {}, sum[4] = {};
        const int e = e0 + 4 * lane;
#pragma unroll 10
        for (int b = warp; b < runs; b += warps) {
            const uint2 n = e < E ? *reinterpret_cast<const uint2 *>(a.counts + static_cast<int64_t>(b) * row + e)
                                  : make_uint2(0, 0);
            const int in = b < first ? 1 : 0, v[4] = {static_cast<int>(n.x & 0xffffu), static_cast<int>(n.x >> 16),
                                                      static_cast<int>(n.y & 0xffffu), static_cast<int>(n.y >> 16)};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                sum[c] += v[c];
                before[c] += in * v[c];
            }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (e + c < E && sum[c]) {
                atomicAdd(&total[e + c], sum[c]);
                atomicAdd(&base[e + c], before[c]);
            }
    }
    __syncthreads();
    if (warp == 0) {
        const int n = add_expert_prefix(a, base, total);
        if (lane == 0)
            used = n;
    }
    __syncthreads();
    rank_pairs(a, p0, p1, pairs, base, wc);
    // rows that no pair takes
    for (int64_t i = used + blockIdx.x * 1024ll + threadIdx.x; i < all; i += gridDim.x * 1024ll)
        a.rows[i] = -1;
}

// Gradient of the weights.  With the softmax over the selected logits,
// dlogit_j = w_j (dw_j - sum_i w_i dw_i) at the selected ones and 0 elsewhere;
// with the softmax p over all, dlogit_e = p_e ([e selected] dw - sum_i p_i dw_i).
template <int C>
__global__ void __launch_bounds__(256)
    route_backward_kernel(const void *logits, bool bf16, int64_t T, int64_t ld, int E, int k, bool normalize,
                          const int32_t *experts, const float *dweights, void *out)
{
    const int lane = threadIdx.x % 32;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x / 32);
    grid_release();
    grid_wait();
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
        float d[C];
#pragma unroll
        for (int c = 0; c < C; ++c)
            d[c] = !normalize && v[c] != 0.f ? -(v[c] / sum) * mean : 0.f;
        for (int j = 0; j < k; ++j) {
            const int ej = __shfl_sync(kFull, e, j);
            const float gj = __shfl_sync(kFull, g, j);
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (ej == lane + 32 * c)
                    d[c] += gj;
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = lane + 32 * c;
            if (i < E) {
                if (bf16)
                    static_cast<__nv_bfloat16 *>(out)[t * E + i] = __float2bfloat16_rn(d[c]);
                else
                    static_cast<float *>(out)[t * E + i] = d[c];
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

// The same as eight packed bf16.
template <bool VEC>
__device__ __forceinline__ uint4 load_packed8(const __nv_bfloat16 *row, int64_t h, int64_t H)
{
    if constexpr (VEC) {
        return *reinterpret_cast<const uint4 *>(row + h);
    } else {
        float f[8];
        load8<false>(row, h, H, f);
        return pack8(f);        // bf16 values: exact
    }
}

// Both kernels are bound by HBM: every Y row is read or written once.  A thread
// keeps the k rows' loads of its eight columns in flight together (KMAX: the
// next of 2, 4, 8, 16 choices).  8191 tokens of 8 choices, 4096 columns: 104 -
// 109 us (6.2 - 6.5 TB/s, of measured 6.8), the gradient 169 - 172 (6.6 - 6.8 TB/s).
constexpr int kCombineThreads = 128;

template <bool VEC, int KMAX>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(CombineArgs a, int64_t parts)
{
    const int64_t t = blockIdx.x / parts;
    const int64_t h = ((blockIdx.x % parts) * kCombineThreads + threadIdx.x) * 8;
    grid_release();
    grid_wait();
    if (h >= a.H)
        return;
    int32_t slot[KMAX];
    float w[KMAX], acc[8] = {};
    uint4 y[KMAX];
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
        const int32_t at = j < a.k ? a.slots[t * a.k + j] : -1;
        slot[j] = at < a.R ? at : -1;
        w[j] = j < a.k && a.weights ? a.weights[t * a.k + j] : 1.f;
    }
    if (a.residual)
        load8<VEC>(static_cast<const __nv_bfloat16 *>(a.residual) + t * a.ldr, h, a.H, acc);
#pragma unroll
    for (int j = 0; j < KMAX; ++j)
        if (slot[j] >= 0)
            y[j] = load_packed8<VEC>(static_cast<const __nv_bfloat16 *>(a.Y) + slot[j] * a.ldy, h, a.H);
#pragma unroll
    for (int j = 0; j < KMAX; ++j)
        if (slot[j] >= 0) {
            float f[8];
            unpack8(y[j], f);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                acc[i] = fmaf(w[j], f[i], acc[i]);
        }
    store8<VEC>(static_cast<__nv_bfloat16 *>(a.out) + t * a.ldo, h, a.H, acc);
}

template <bool VEC, int KMAX>
__global__ void __launch_bounds__(256) combine_backward_kernel(CombineGradArgs a)
{
    __shared__ float part[8][KMAX];
    const int64_t t = blockIdx.x;
    grid_release();
    grid_wait();
    int32_t slot[KMAX];
    float w[KMAX], dot[KMAX];
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
        const int32_t s = j < a.k ? a.slots[t * a.k + j] : -1;
        slot[j] = s < a.R ? s : -1;
        w[j] = j < a.k && a.weights ? a.weights[t * a.k + j] : 1.f;
        dot[j] = 0.f;
    }
    const __nv_bfloat16 *Y = static_cast<const __nv_bfloat16 *>(a.Y);
    __nv_bfloat16 *dY = static_cast<__nv_bfloat16 *>(a.dY);
    for (int64_t h = threadIdx.x * 8; h < a.H; h += 256 * 8) {
        float d[8];
        uint4 y[KMAX];
        load8<VEC>(static_cast<const __nv_bfloat16 *>(a.dOut) + t * a.ldo, h, a.H, d);
        if (a.dweights) {
#pragma unroll
            for (int j = 0; j < KMAX; ++j)
                if (slot[j] >= 0)
                    y[j] = load_packed8<VEC>(Y + slot[j] * a.ldy, h, a.H);
        }
#pragma unroll
        for (int j = 0; j < KMAX; ++j)
            if (slot[j] >= 0) {
                float o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    o[i] = w[j] * d[i];
                store8<VEC>(dY + slot[j] * a.H, h, a.H, o);
            }
        if (a.dweights) {
#pragma unroll
            for (int j = 0; j < KMAX; ++j)
                if (slot[j] >= 0) {
                    float f[8];
                    unpack8(y[j], f);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        dot[j] = fmaf(d[i], f[i], dot[j]);
                }
        }
    }
    if (!a.dweights)
        return;
#pragma unroll
    for (int j = 0; j < KMAX; ++j) {
        const float v = warp_sum(dot[j]);
        if (threadIdx.x % 32 == 0)
            part[threadIdx.x / 32][j] = v;
    }
    __syncthreads();
    if (threadIdx.x < a.k) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v += part[i][threadIdx.x];
        a.dweights[t * a.k + threadIdx.x] = v;
    }
}

constexpr int64_t kOneBlockTokens = 128;

// Runs of tokens: two per SM, and at most 4095 tokens, so that a run's counts
// fit 16 bits.
int tokens_per_run(int64_t T, int num_sms)
{
    return static_cast<int>(std::min<int64_t>((T + 2 * num_sms - 1) / (2 * num_sms), 4095));
}

int route_runs(int64_t T, int num_sms)
{
    const int each = tokens_per_run(T, num_sms);
    return static_cast<int>((T + each - 1) / each);
}

// Dynamic shared memory above the default limit needs an attribute.
cudaError_t smem_limit(const void *kern, int bytes) { return bytes > 48 * 1024 ? ensure_smem_attr(kern, bytes) : cudaSuccess; }

template <int C, bool BF16>
cudaError_t launch_route_as(const RouteArgs &a, int num_sms, cudaStream_t s)
{
    cudaError_t e;
    if (a.T <= kOneBlockTokens) {
        // a warp per token; fewer counters where there are fewer tokens
        const int warps = static_cast<int>(a.T < 4 ? 4 : a.T < 16 ? a.T : 16);
        const int bytes = static_cast<int>(((2 + warps) * a.E + a.T * a.k) * sizeof(int32_t));
        if ((e = smem_limit(reinterpret_cast<const void *>(route_one_kernel<C, BF16>), bytes)) != cudaSuccess)
            return e;
        return launch_overlapped(route_one_kernel<C, BF16>, dim3(1), warps * 32, bytes, 1, s, a);
    }
    const int each = tokens_per_run(a.T, num_sms), runs = route_runs(a.T, num_sms);
    if ((e = launch_overlapped(route_choose_kernel<C, BF16>, dim3(runs), 1024, a.E * sizeof(int32_t), 1, s, a, each)) !=
        cudaSuccess)
        return e;
    const int span = 2 * each * a.k, bytes = static_cast<int>((34 * a.E + (span <= kPlanPairs ? span : 0)) * sizeof(int32_t));
    if ((e = smem_limit(reinterpret_cast<const void *>(route_plan_kernel), bytes)) != cudaSuccess)
        return e;
    return launch_overlapped(route_plan_kernel, dim3((runs + 1) / 2), 1024, bytes, 1, s, a, each, runs);
}

template <int C>
cudaError_t launch_route_of(const RouteArgs &a, int num_sms, cudaStream_t s)
{
    return a.bf16 ? launch_route_as<C, true>(a, num_sms, s) : launch_route_as<C, false>(a, num_sms, s);
}

bool vec8(const void *p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 8 == 0; }

}  // namespace

size_t route_counts_bytes(int64_t T, int E, int num_sms)
{
    return static_cast<size_t>(T > kOneBlockTokens ? route_runs(T, num_sms) : 1) * count_row(E) * sizeof(uint16_t);
}

// Registers per lane for E experts: 2, 4, 8 or 32 of 32 experts each.
cudaError_t launch_route(const RouteArgs &a, int num_sms, cudaStream_t s)
{
    return a.E <= 64    ? launch_route_of<2>(a, num_sms, s)
           : a.E <= 128 ? launch_route_of<4>(a, num_sms, s)
           : a.E <= 256 ? launch_route_of<8>(a, num_sms, s)
                        : launch_route_of<32>(a, num_sms, s);
}

cudaError_t launch_route_backward(const void *logits, bool bf16, int64_t T, int64_t ld, int E, int k, bool normalize,
                                  const int32_t *experts, const float *dweights, void *dlogits, int num_sms,
                                  cudaStream_t s)
{
    const int blocks = static_cast<int>(std::min<int64_t>((T + 7) / 8, num_sms * 32));
    auto kern = E <= 64    ? route_backward_kernel<2>
                : E <= 128 ? route_backward_kernel<4>
                : E <= 256 ? route_backward_kernel<8>
                           : route_backward_kernel<32>;
    return launch_overlapped(kern, dim3(blocks), 256, 0, 1, s, logits, bf16, T, ld, E, k, normalize, experts, dweights, dlogits);
}

cudaError_t launch_combine(const CombineArgs &a, cudaStream_t s)
{
    const int64_t parts = (a.H + kCombineThreads * 8 - 1) / (kCombineThreads * 8);
    const bool vec = a.H % 8 == 0 && vec8(a.Y, a.ldy) && vec8(a.out, a.ldo) && (!a.residual || vec8(a.residual, a.ldr));
    auto kern = a.k <= 2   ? (vec ? combine_kernel<true, 2> : combine_kernel<false, 2>)
                : a.k <= 4 ? (vec ? combine_kernel<true, 4> : combine_kernel<false, 4>)
                : a.k <= 8 ? (vec ? combine_kernel<true, 8> : combine_kernel<false, 8>)
                           : (vec ? combine_kernel<true, 16> : combine_kernel<false, 16>);
    return launch_overlapped(kern, dim3(static_cast<unsigned>(a.T * parts)), kCombineThreads, 0, 1, s, a, parts);
}

cudaError_t launch_combine_backward(const CombineGradArgs &a, cudaStream_t s)
{
    const bool vec = a.H % 8 == 0 && vec8(a.Y, a.ldy) && vec8(a.dOut, a.ldo) && vec8(a.dY, a.H);
    auto kern = a.k <= 2   ? (vec ? combine_backward_kernel<true, 2> : combine_backward_kernel<false, 2>)
                : a.k <= 4 ? (vec ? combine_backward_kernel<true, 4> : combine_backward_kernel<false, 4>)
                : a.k <= 8 ? (vec ? combine_backward_kernel<true, 8> : combine_backward_kernel<false, 8>)
                           : (vec ? combine_backward_kernel<true, 16> : combine_backward_kernel<false, 16>);
    return launch_overlapped(kern, dim3(static_cast<unsigned>(a.T)), 256, 0, 1, s, a);
}

}  // namespace tmg
