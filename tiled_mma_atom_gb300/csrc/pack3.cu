// pack3.cu — operands of the grouped and the dense products that TMA cannot
// read in place (unaligned or broadcast rows, strides in both directions, an
// empty contraction) copied to workspace: dst[e][r][k], rows of Kp elements,
// zero-padded past `rows` and K.  32 x 32 tiles through shared memory: reads
// run along the source's smaller stride, writes along k.
#include "grouped.h"

namespace tmg {
namespace {

template <typename T>
__global__ void __launch_bounds__(256) pack3_kernel(Pack3Args a, int64_t tiles_k, int64_t tiles_r)
{
    __shared__ T t[32][33];
    const T *src = static_cast<const T *>(a.src);
    T *dst = static_cast<T *>(a.dst);
    const int x = threadIdx.x % 32, y = threadIdx.x / 32;
    const bool along_rows = a.s_row < a.s_col;
    for (int64_t i = blockIdx.x; i < tiles_k * tiles_r * a.E; i += gridDim.x) {
        const int64_t k0 = i % tiles_k * 32, r0 = i / tiles_k % tiles_r * 32, e = i / (tiles_k * tiles_r);
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
            const int64_t r = r0 + (along_rows ? x : y + j), k = k0 + (along_rows ? y + j : x);
            const T v = r < a.rows && k < a.K ? src[e * a.s_e + r * a.s_row + k * a.s_col] : T(0);
            t[along_rows ? x : y + j][along_rows ? y + j : x] = v;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 32; j += 8)
            if (r0 + y + j < a.rows_p && k0 + x < a.Kp)
                dst[e * a.d_e + (r0 + y + j) * a.Kp + k0 + x] = t[y + j][x];
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_pack3(const Pack3Args &a, int elem, int num_sms, cudaStream_t s)
{
    const int64_t tk = (a.Kp + 31) / 32, tr = (a.rows_p + 31) / 32, total = tk * tr * a.E;
    if (total == 0)
        return cudaSuccess;
    const unsigned blocks = static_cast<unsigned>(total < num_sms * 8 ? total : num_sms * 8);
    note_launch();
    if (elem == 1)
        pack3_kernel<uint8_t><<<blocks, 256, 0, s>>>(a, tk, tr);
    else
        pack3_kernel<uint16_t><<<blocks, 256, 0, s>>>(a, tk, tr);
    return cudaGetLastError();
}

}  // namespace tmg
