// pack3.cu — operands of the grouped and the dense products that TMA cannot
// read in place (unaligned or broadcast rows, strides in both directions, an
// empty contraction) copied to workspace: dst[e][r][k], rows of Kp elements,
// zero-padded past `rows` and K.  Contiguous rows in 16-byte pieces, others in
// 32 x 32 tiles through shared memory: reads run along the source's smaller
// stride, writes along k.  And the gather of
// rows by number, for products whose tiles are too wide for TMA gathers.
#include "grouped.h"
#include "launch.cuh"

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
    grid_release();
    grid_wait();
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

// The same for rows of contiguous elements (less than 2^31 pieces): a thread makes
// 16-byte pieces of dst, four in flight, read in words of the widest type that
// the source's address and strides are multiples of (weight gradient of 8191 rows,
// 4100 x 4100, both operands copied: 386 us through the tiles above, 265 so).
template <typename W>
__global__ void __launch_bounds__(256) pack_rows_kernel(Pack3Args a, int elem, uint32_t pieces)
{
    constexpr int kWords = 16 / sizeof(W), kPieces = 4;
    const int64_t bytes = a.K * elem;
    const uint32_t per = static_cast<uint32_t>(a.Kp * elem / 16), rows_p = static_cast<uint32_t>(a.rows_p);
    const uint32_t step = gridDim.x * 256u;
    grid_release();
    grid_wait();
    for (uint32_t i0 = blockIdx.x * 256u + threadIdx.x; i0 < pieces; i0 += kPieces * step) {
        union {
            uint4 v;
            W w[kWords];
            uint8_t b[16];
        } u[kPieces];
#pragma unroll
        for (int h = 0; h < kPieces; ++h) {
            const uint32_t i = i0 + h * step, row = i / per, e = row / rows_p, r = row - e * rows_p;
            const int64_t at = (i - row * per) * 16ll;
            const char *p = static_cast<const char *>(a.src) + (e * a.s_e + r * a.s_row) * elem + at;
            u[h].v = make_uint4(0, 0, 0, 0);
            if (i < pieces && r < a.rows) {
                if (at + 16 <= bytes) {
#pragma unroll
                    for (int j = 0; j < kWords; ++j)
                        u[h].w[j] = reinterpret_cast<const W *>(p)[j];
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (at + j < bytes)
                            u[h].b[j] = p[j];
                }
            }
        }
#pragma unroll
        for (int h = 0; h < kPieces; ++h) {
            const uint32_t i = i0 + h * step, row = i / per, e = row / rows_p, r = row - e * rows_p;
            if (i < pieces)
                *reinterpret_cast<uint4 *>(static_cast<char *>(a.dst) + (e * a.d_e + r * a.Kp) * elem + (i - row * per) * 16ll) =
                    u[h].v;
        }
    }
}

// Rows in 16-byte pieces: dst[r] = src[numbers[r]], zeros where that is no row
// and past the row's bytes.  A warp takes a row at a time, eight pieces per
// lane in flight.
__global__ void __launch_bounds__(256)
    gather_rows_kernel(const char *src, int64_t stride, int64_t src_rows, int64_t bytes, const int32_t *numbers, int64_t rows,
                       char *dst, int64_t dst_stride)
{
    const int lane = threadIdx.x % 32, pieces = static_cast<int>(dst_stride / 16), whole = static_cast<int>(bytes / 16), tail = static_cast<int>(bytes % 16);
    grid_release();
    grid_wait();
    for (int64_t r = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / 32; r < rows; r += gridDim.x * 8ll) {
        const int64_t from = numbers[r];
        const bool there = from >= 0 && from < src_rows;
        const char *p = src + (there ? from : 0) * stride;
        uint4 *d = reinterpret_cast<uint4 *>(dst + r * dst_stride);
        for (int i = lane; i < pieces; i += 256) {
            uint4 v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int at = i + 32 * j;
                v[j] = there && at < whole ? reinterpret_cast<const uint4 *>(p)[at] : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (i + 32 * j < pieces)
                    d[i + 32 * j] = v[j];
        }
        __syncwarp();
        // the last, partial piece
        if (there && whole < pieces && lane < tail)
            reinterpret_cast<char *>(d + whole)[lane] = p[bytes - tail + lane];
    }
}

}  // namespace

cudaError_t launch_gather_rows(const void *src, int64_t stride, int64_t src_rows, int64_t bytes, const int32_t *numbers,
                               int64_t rows, void *dst, int64_t dst_stride, int num_sms, cudaStream_t s)
{
    const int64_t blocks = (rows + 7) / 8;
    if (rows == 0)
        return cudaSuccess;
    return launch_overlapped(gather_rows_kernel, dim3(static_cast<unsigned>(blocks < num_sms * 8 ? blocks : num_sms * 8)), 256, 0,
                             1, s, static_cast<const char *>(src), stride, src_rows, bytes, numbers, rows,
                             static_cast<char *>(dst), dst_stride);
}

cudaError_t launch_pack3(const Pack3Args &a, int elem, int num_sms, cudaStream_t s)
{
    const int64_t tk = (a.Kp + 31) / 32, tr = (a.rows_p + 31) / 32, total = tk * tr * a.E;
    if (total == 0)
        return cudaSuccess;
    const int64_t pieces = a.E * a.rows_p * (a.Kp * elem / 16);
    if ((a.s_col == 1 || a.K == 1) && pieces < (int64_t{1} << 31)) {
        const int64_t need = (pieces + 255) / 256;
        const unsigned grid = static_cast<unsigned>(need < num_sms * 8 ? need : num_sms * 8);
        const uint64_t align = reinterpret_cast<uintptr_t>(a.src) | static_cast<uint64_t>(a.s_row * elem) |
                               static_cast<uint64_t>(a.s_e * elem);
        auto *k = align % 8 == 0   ? pack_rows_kernel<unsigned long long>
                  : align % 4 == 0 ? pack_rows_kernel<unsigned>
                  : align % 2 == 0 ? pack_rows_kernel<unsigned short>
                                   : pack_rows_kernel<unsigned char>;
        return launch_overlapped(k, dim3(grid), 256, 0, 1, s, a, elem, static_cast<uint32_t>(pieces));
    }
    const unsigned blocks = static_cast<unsigned>(total < num_sms * 8 ? total : num_sms * 8);
    return launch_overlapped(elem == 1 ? pack3_kernel<uint8_t> : pack3_kernel<uint16_t>, dim3(blocks), 256, 0, 1, s, a, tk, tr);
}

}  // namespace tmg
