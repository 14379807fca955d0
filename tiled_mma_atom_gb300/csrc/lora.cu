// lora.cu — the low-rank side of dense projections with adapters: a row's product
// with its adapter's first factor, the way back through the second, and the
// factors' gradients.
#include <cuda_bf16.h>

#include "launch.cuh"
#include "lora.h"

namespace tmg {
namespace {

__device__ __forceinline__ float bf(const void *p, int64_t i) { return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]); }

constexpr int kThreads = 256;

// A block per row; a warp per rank (F's rows along c), or threads over ranks and
// slices of c (`across`), summed in slice order.
__global__ void __launch_bounds__(kThreads) rank_kernel(RankArgs a)
{
    __shared__ float part[kThreads];
    grid_release();
    grid_wait();
    const int64_t m = blockIdx.x;
    const int l = a.adapters[m];
    const bool on = l >= 0 && l < a.L;
    const float scale = on && a.scales ? a.scales[l] : 1.f;
    __nv_bfloat16 *U = static_cast<__nv_bfloat16 *>(a.U) + m * a.ldu;
    const int64_t f0 = on ? l * a.C * a.r : 0, x0 = m * a.ldx;
    if (!on) {
        for (int j = threadIdx.x; j < a.r; j += kThreads)
            U[j] = __float2bfloat16_rn(0.f);
    } else if (!a.across) {
        for (int j = threadIdx.x / 32; j < a.r; j += kThreads / 32) {
            float sum = 0.f;
            for (int64_t c = threadIdx.x % 32; c < a.C; c += 32)
                sum = fmaf(bf(a.X, x0 + c), bf(a.F, f0 + j * a.C + c), sum);
#pragma unroll
            for (int o = 16; o; o >>= 1)
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (threadIdx.x % 32 == 0)
                U[j] = __float2bfloat16_rn(scale * sum);
        }
    } else {
        const int slices = kThreads / a.r, j = threadIdx.x % a.r, slice = threadIdx.x / a.r;
        float sum = 0.f;
        if (slice < slices)
            for (int64_t c = slice; c < a.C; c += slices)
                sum = fmaf(bf(a.X, x0 + c), bf(a.F, f0 + c * a.r + j), sum);
        part[threadIdx.x] = sum;
        __syncthreads();
        if (threadIdx.x < a.r) {
            sum = 0.f;
            for (int i = 0; i < slices; ++i)
                sum += part[i * a.r + threadIdx.x];
            U[threadIdx.x] = __float2bfloat16_rn(scale * sum);
        }
    }
}

}  // namespace

cudaError_t launch_lora_rank(const RankArgs &a, cudaStream_t s)
{
    return launch_overlapped(rank_kernel, dim3(static_cast<unsigned>(a.M)), kThreads, 0, 1, s, a);
}

}  // namespace tmg
