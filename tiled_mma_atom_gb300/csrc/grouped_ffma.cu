// grouped_ffma.cu — the expert-grouped products on CUDA cores, for operands
// of any strides: 64 x 64 output tiles, 256 threads with 4 x 4 fp32
// accumulators each, 16 contraction elements staged in shared memory at a
// time.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "act.cuh"
#include "grouped.h"

namespace tmg {
namespace {

constexpr int kT = 64, kC = 16;

__device__ __forceinline__ float read_elem(const void *p, int64_t i, bool e4m3)
{
    if (e4m3)
        return static_cast<float>(static_cast<const __nv_fp8_e4m3 *>(p)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

// Group bounds clamped to the R rows there are, so that no offset can lead
// outside the buffers.
__device__ __forceinline__ void group_range(const int32_t *offsets, int64_t e, int64_t R, int64_t &lo, int64_t &hi)
{
    lo = 0;
    hi = R;
    if (offsets) {
        lo = min(max(static_cast<int64_t>(offsets[e]), int64_t{0}), R);
        hi = min(max(static_cast<int64_t>(offsets[e + 1]), lo), R);
    }
}

__device__ __forceinline__ float act_rt(float z, int act)
{
    switch (act) {
    case kActRelu: return act_f<kActRelu>(z);
    case kActSilu: return act_f<kActSilu>(z);
    case kActGelu: return act_f<kActGelu>(z);
    default: return z;
    }
}

__global__ void __launch_bounds__(256) grouped_ffma_kernel(GroupedArgs a, int64_t a_col)
{
    __shared__ float sa[kC][kT + 1], sb[2][kC][kT + 1];
    const int64_t e = blockIdx.z, nout = a.out_n();
    int64_t lo, hi;
    group_range(a.offsets, e, a.R, lo, hi);
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    const bool two = a.epi.act == kActSwiglu;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kT;
    for (int64_t r0 = lo + static_cast<int64_t>(blockIdx.y) * kT; r0 < hi; r0 += static_cast<int64_t>(gridDim.y) * kT) {
        float acc[2][4][4] = {};
        for (int64_t k0 = 0; k0 < a.K; k0 += kC) {
            for (int i = threadIdx.x; i < kC * kT; i += 256) {
                const int c = i % kC, t = i / kC;
                const int64_t k = k0 + c, r = r0 + t, n = n0 + t;
                float va = 0.f, vb = 0.f, vu = 0.f;
                if (k < a.K && r < hi) {
                    const int64_t src = a.rows ? a.rows[r] : r;
                    if (src >= 0 && src < a.T)
                        va = read_elem(a.A, src * a.lda + k * a_col, a.e4m3);
                }
                if (k < a.K && n < nout) {
                    vb = read_elem(a.B, e * a.b_expert + n * a.b_row + k * a.b_col, a.e4m3);
                    if (two)
                        vu = read_elem(a.B, e * a.b_expert + (nout + n) * a.b_row + k * a.b_col, a.e4m3);
                }
                sa[c][t] = va;
                sb[0][c][t] = vb;
                sb[1][c][t] = vu;
            }
            __syncthreads();
            for (int c = 0; c < kC; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        acc[0][i][j] = fmaf(sa[c][ty + 16 * i], sb[0][c][tx + 16 * j], acc[0][i][j]);
                        acc[1][i][j] = fmaf(sa[c][ty + 16 * i], sb[1][c][tx + 16 * j], acc[1][i][j]);
                    }
            __syncthreads();
        }
        __nv_bfloat16 *D = static_cast<__nv_bfloat16 *>(a.D);
        __nv_bfloat16 *P = static_cast<__nv_bfloat16 *>(a.epi.preact);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t r = r0 + ty + 16 * i;
            if (r >= hi)
                continue;
            float scale = 1.f;
            if (a.epi.scale_a) {
                const int64_t src = a.rows ? a.rows[r] : r;
                scale = src >= 0 && src < a.T ? a.epi.scale_a[src] : 0.f;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t n = n0 + tx + 16 * j;
                if (n >= nout)
                    continue;
                float z = acc[0][i][j] * scale;
                if (a.epi.scale_b)
                    z *= a.epi.scale_b[e * a.N + n];
                if (two) {
                    float u = acc[1][i][j] * scale;
                    if (a.epi.scale_b)
                        u *= a.epi.scale_b[e * a.N + nout + n];
                    if (P) {
                        P[r * a.epi.ld_preact + n] = __float2bfloat16_rn(z);
                        P[r * a.epi.ld_preact + nout + n] = __float2bfloat16_rn(u);
                    }
                    D[r * a.ldd + n] = __float2bfloat16_rn(silu_f(z) * u);
                } else if (a.epi.act == kActSwigluGrad) {
                    float dg, du;
                    swiglu_grad(z, __bfloat162float(P[r * a.epi.ld_preact + n]),
                                __bfloat162float(P[r * a.epi.ld_preact + nout + n]), dg, du);
                    D[r * a.ldd + n] = __float2bfloat16_rn(dg);
                    D[r * a.ldd + nout + n] = __float2bfloat16_rn(du);
                } else {
                    if (a.epi.bias)
                        z += a.epi.bias[n];
                    if (P)
                        P[r * a.epi.ld_preact + n] = __float2bfloat16_rn(z);
                    z = act_rt(z, a.epi.act);
                    if (a.epi.residual)
                        z += __bfloat162float(
                            static_cast<const __nv_bfloat16 *>(a.epi.residual)[r * a.epi.ld_residual + n]);
                    D[r * a.ldd + n] = __float2bfloat16_rn(z);
                }
            }
        }
    }
}

__global__ void __launch_bounds__(256) wgrad_ffma_kernel(WgradArgs a, int64_t d_col, int64_t a_col)
{
    __shared__ float sd[kC][kT + 1], sa[kC][kT + 1];
    const int64_t e = blockIdx.z, n0 = static_cast<int64_t>(blockIdx.y) * kT, k0 = static_cast<int64_t>(blockIdx.x) * kT;
    int64_t lo, hi;
    group_range(a.offsets, e, a.R, lo, hi);
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[4][4] = {};
    for (int64_t r0 = lo; r0 < hi; r0 += kC) {
        for (int i = threadIdx.x; i < kC * kT; i += 256) {
            const int c = i / kT, t = i % kT;
            const int64_t r = r0 + c;
            float vd = 0.f, va = 0.f;
            if (r < hi) {
                if (n0 + t < a.N)
                    vd = read_elem(a.dD, r * a.ldd + (n0 + t) * d_col, false);
                const int64_t src = a.rows ? a.rows[r] : r;
                if (k0 + t < a.K && src >= 0 && src < a.T)
                    va = read_elem(a.A, src * a.lda + (k0 + t) * a_col, false);
            }
            sd[c][t] = vd;
            sa[c][t] = va;
        }
        __syncthreads();
        for (int c = 0; c < kC; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = fmaf(sd[c][ty + 16 * i], sa[c][tx + 16 * j], acc[i][j]);
        __syncthreads();
    }
    __nv_bfloat16 *dB = static_cast<__nv_bfloat16 *>(a.dB) + e * a.N * a.K;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t n = n0 + ty + 16 * i, k = k0 + tx + 16 * j;
            if (n < a.N && k < a.K)
                dB[n * a.K + k] = __float2bfloat16_rn(acc[i][j]);
        }
}

}  // namespace

cudaError_t launch_grouped_ffma(const GroupedArgs &a, int64_t a_col, const ErrCtx &err, cudaStream_t s)
{
    (void)err;
    // row tiles of an evenly filled group, each block walking on where its
    // group is larger
    int64_t tiles = (a.R / a.E + kT) / kT;
    tiles = tiles > 4096 ? 4096 : tiles;
    note_launch();
    grouped_ffma_kernel<<<dim3(static_cast<unsigned>((a.out_n() + kT - 1) / kT), static_cast<unsigned>(tiles),
                               static_cast<unsigned>(a.E)),
                          256, 0, s>>>(a, a_col);
    return cudaGetLastError();
}

cudaError_t launch_wgrad_ffma(const WgradArgs &a, int64_t d_col, int64_t a_col, const ErrCtx &err, cudaStream_t s)
{
    (void)err;
    note_launch();
    wgrad_ffma_kernel<<<dim3(static_cast<unsigned>((a.K + kT - 1) / kT), static_cast<unsigned>((a.N + kT - 1) / kT),
                             static_cast<unsigned>(a.E)),
                        256, 0, s>>>(a, d_col, a_col);
    return cudaGetLastError();
}

}  // namespace tmg
