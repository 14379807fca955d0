// act_grad.cu — the elementwise part of the dense product's gradient:
// dz = dD act'(z) rounded to bf16 for the two products that follow, and the
// bias gradient, the column sums of the fp32 dz (before that rounding), added
// up in a fixed order: rows of a chunk by one thread, then the chunks.
//
// dz is rounded because the products' tensor instructions take bf16: dA and dB are
// then off by 0.0023 of their size, against 0.0017 with dz held in fp32 (8191 x 4096
// x 4096, GELU; the results' own rounding is 0.0017 of it).  With activation none dz
// is dD itself and nothing is rounded.
//
// Bound by its 6 bytes an element.  A thread keeps four rows' loads in flight:
// with one, the gradient of an 8191 x 4096 x 4096 product with GELU (dz 41 us of
// it) took 347 us and takes 342.
#include <cuda_bf16.h>

#include "act.cuh"
#include "grouped.h"
#include "launch.cuh"

namespace tmg {
namespace {

constexpr int kCols = 256;    // a block: 32 threads x 8 columns, 8 row lanes, 4 rows of each in flight

// Rows of a chunk: 128, or 32 where that leaves few blocks (gradient of 158 x 7544 x
// 6088 with GELU 86.2 us with 128, 77.4 with 32).
int chunk_rows(int64_t M, int64_t N) { return (M + 127) / 128 * ((N + kCols - 1) / kCols) >= 512 ? 128 : 32; }

template <int ACT, bool VEC>
__global__ void __launch_bounds__(256)
    act_grad_kernel(const __nv_bfloat16 *dD, int64_t ldd, const __nv_bfloat16 *Z, int64_t ldp, int64_t M, int64_t N, int chunk,
                    int chunks, __nv_bfloat16 *dz, float *partials)
{
    __shared__ float red[8][kCols];
    grid_release();
    grid_wait();
    const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x / chunks) * kCols, c = n0 + tx * 8;
    const int64_t row = blockIdx.x % chunks, m0 = row * chunk;
    float sum[8] = {};
    const int64_t m1 = min(M, m0 + chunk);
    if (VEC && c < N) {
        for (int64_t m = m0 + ty; m < m1; m += 32) {
            uint4 d[4], z[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const bool in = m + 8 * r < m1;
                d[r] = in ? *reinterpret_cast<const uint4 *>(dD + (m + 8 * r) * ldd + c) : make_uint4(0, 0, 0, 0);
                if constexpr (ACT != kActNone)
                    z[r] = in ? *reinterpret_cast<const uint4 *>(Z + (m + 8 * r) * ldp + c) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if (m + 8 * r >= m1)
                    break;
                const uint32_t du[4] = {d[r].x, d[r].y, d[r].z, d[r].w};
                uint32_t zu[4] = {}, ou[4];
                if constexpr (ACT != kActNone)
                    zu[0] = z[r].x, zu[1] = z[r].y, zu[2] = z[r].z, zu[3] = z[r].w;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float a = __uint_as_float(du[i] << 16) * act_grad<ACT>(__uint_as_float(zu[i] << 16));
                    const float b = __uint_as_float(du[i] & 0xffff0000u) * act_grad<ACT>(__uint_as_float(zu[i] & 0xffff0000u));
                    sum[2 * i] += a;
                    sum[2 * i + 1] += b;
                    ou[i] = pack_bf16x2(a, b);
                }
                if (dz)
                    *reinterpret_cast<uint4 *>(dz + (m + 8 * r) * N + c) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
            }
        }
    } else if (!VEC) {
        for (int64_t m = m0 + ty; m < m1; m += 8) {
            float v[8], z[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = c + i < N ? __bfloat162float(dD[m * ldd + c + i]) : 0.f;
                if constexpr (ACT != kActNone)
                    z[i] = c + i < N ? __bfloat162float(Z[m * ldp + c + i]) : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if constexpr (ACT != kActNone)
                    v[i] *= act_grad<ACT>(z[i]);
                sum[i] += v[i];
                if (dz && c + i < N)
                    dz[m * N + c + i] = __float2bfloat16_rn(v[i]);
            }
        }
    }
    if (!partials)
        return;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        red[ty][tx * 8 + i] = sum[i];
    __syncthreads();
    const int64_t n = n0 + threadIdx.x;
    if (n < N) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w)
            v += red[w][threadIdx.x];
        partials[row * N + n] = v;
    }
}

__global__ void __launch_bounds__(256)
    column_sum_kernel(const float *partials, int chunks, int64_t N, float *out)
{
    __shared__ float red[8][32];
    grid_release();
    grid_wait();
    const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
    const int64_t n = static_cast<int64_t>(blockIdx.x) * 32 + tx;
    float v = 0.f;
    if (n < N)
        for (int i = ty; i < chunks; i += 8)
            v += partials[static_cast<int64_t>(i) * N + n];
    red[ty][tx] = v;
    __syncthreads();
    if (ty == 0 && n < N) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w)
            s += red[w][tx];
        out[n] = s;
    }
}

template <int ACT>
cudaError_t launch_act(const void *dD, int64_t ldd, const void *Z, int64_t ldp, int64_t M, int64_t N, void *dz,
                       float *partials, cudaStream_t s)
{
    auto ok = [](const void *p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 8 == 0; };
    const bool vec = N % 8 == 0 && ok(dD, ldd) && (ACT == kActNone || ok(Z, ldp)) && ok(dz, N);
    // one dimension: wide results have more column blocks than a grid's second may
    const int chunks = act_grad_chunks(M, N);
    const dim3 grid(static_cast<unsigned>(chunks * ((N + kCols - 1) / kCols)));
    const __nv_bfloat16 *d = static_cast<const __nv_bfloat16 *>(dD), *z = static_cast<const __nv_bfloat16 *>(Z);
    return launch_overlapped(vec ? act_grad_kernel<ACT, true> : act_grad_kernel<ACT, false>, grid, 256, 0, 1, s, d, ldd, z, ldp, M,
                             N, chunk_rows(M, N), chunks, static_cast<__nv_bfloat16 *>(dz), partials);
}

}  // namespace

int act_grad_chunks(int64_t M, int64_t N) { return static_cast<int>((M + chunk_rows(M, N) - 1) / chunk_rows(M, N)); }

cudaError_t launch_act_grad(const void *dD, int64_t ldd, const void *preact, int64_t ldp, int act, int64_t M, int64_t N,
                            void *dz, float *partials, float *dbias, cudaStream_t s)
{
    cudaError_t e;
    switch (act) {
    case kActRelu: e = launch_act<kActRelu>(dD, ldd, preact, ldp, M, N, dz, dbias ? partials : nullptr, s); break;
    case kActSilu: e = launch_act<kActSilu>(dD, ldd, preact, ldp, M, N, dz, dbias ? partials : nullptr, s); break;
    case kActGelu: e = launch_act<kActGelu>(dD, ldd, preact, ldp, M, N, dz, dbias ? partials : nullptr, s); break;
    default: e = launch_act<kActNone>(dD, ldd, preact, ldp, M, N, dz, dbias ? partials : nullptr, s); break;
    }
    if (e != cudaSuccess || !dbias)
        return e;
    return launch_overlapped(column_sum_kernel, dim3(static_cast<unsigned>((N + 31) / 32)), 256, 0, 1, s, partials,
                             act_grad_chunks(M, N), N, dbias);
}

}  // namespace tmg
