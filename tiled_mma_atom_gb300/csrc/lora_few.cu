// lora_few.cu — the dense product with low-rank adapters for a few rows (decoding): W
// is read once, every row has an adapter of its own.
//
// First kernel: U[m][j], a warp per (row, rank), 16 bytes of X and F per lane and load.
// Second kernel: W's product as in few.cuh, for which nothing but x is needed, so it
// starts while the first one runs and waits for U only in the warps that add the
// adapters' share: those form U[m] . F[a_m][n] for the results of their CTA, a thread
// per result, while W's blocks come in.  The first kernel lets the second one start
// only after its own wait for the kernel before, so x and the weights are complete
// by then.
//
// Bound by HBM: W and the rows' factors once.
#include <cuda_bf16.h>

#include "few.cuh"
#include "lora.h"

namespace tmg {
namespace {

constexpr int kLfThreads = 384;
constexpr int kLfRanks = 8;                  // ranks (warps) of a block of the first kernel

__device__ __forceinline__ float dot8(const uint4 &a, const uint4 &b, float sum)
{
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        sum = fmaf(__uint_as_float(x[i] << 16), __uint_as_float(y[i] << 16), sum);
        sum = fmaf(__uint_as_float(x[i] & 0xffff0000u), __uint_as_float(y[i] & 0xffff0000u), sum);
    }
    return sum;
}

__global__ void __launch_bounds__(kLfRanks * 32) lora_few_rank_kernel(RankArgs a, int groups)
{
    grid_wait();
    grid_release();
    const int64_t m = blockIdx.x / groups;
    const int j = blockIdx.x % groups * kLfRanks + threadIdx.x / 32, lane = threadIdx.x % 32;
    if (j >= a.r && j >= a.ldu)
        return;
    const int l = a.adapters[m];
    float sum = 0.f;                     // also in the columns past r that pad a row
    if (l >= 0 && l < a.L && j < a.r) {
        const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.X) + m * a.ldx);
        const uint4 *f = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.F) + (static_cast<int64_t>(l) * a.r + j) * a.C);
        const int n = static_cast<int>(a.C / 8);
        for (int c = lane; c < n; c += 256) {
            uint4 v[8], w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool in = c + 32 * i < n;
                v[i] = in ? f[c + 32 * i] : make_uint4(0, 0, 0, 0);
                w[i] = in ? x[c + 32 * i] : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sum = dot8(v[i], w[i], sum);
        }
        if (a.scales)
            sum *= a.scales[l];
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0)
        static_cast<__nv_bfloat16 *>(a.U)[m * a.ldu + j] = __float2bfloat16_rn(sum);
}

__device__ __forceinline__ float ld_cluster_one(uint32_t addr, uint32_t rank)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa_shared(addr, rank)) : "memory");
    return v;
}

__global__ void __launch_bounds__(kLfThreads) lora_few_kernel(const __grid_constant__ LoraFewArgs p, ErrCtx err)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ FewRing sm;
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t *ring = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    float *share = reinterpret_cast<float *>(ring + p.shape.ring_bytes);   // the adapters' share of this CTA's results
    const uint32_t rank = cluster_ctarank(), S = few_cluster_size();
    const int n0 = blockIdx.x / S * 128, num_kb = ceil_div(p.K, 64);
    const int kb0 = static_cast<int>(static_cast<int64_t>(num_kb) * rank / S);
    const int kb1 = static_cast<int>(static_cast<int64_t>(num_kb) * (rank + 1) / S);
    few_setup(p.shape, sm, &p.tmW, &p.tmX);
    grid_release();
    __syncthreads();
    tc_fence_after();
    const int items = p.M * 128, first = items * rank / S, last = items * (rank + 1) / S;
    few_product(
        p.shape, sm, ring, kb0, kb1, [&](uint8_t *dst, uint64_t *bar, int kb) { tma_load_2d_w(dst, &p.tmW, bar, kb * 64, n0); },
        [&](uint8_t *dst, uint64_t *bar, int kb) { tma_load_2d_w(dst, &p.tmX, bar, kb * 64, 0); }, [] {},
        [&] {
            grid_wait();                         // U
            const __nv_bfloat16 *U = static_cast<const __nv_bfloat16 *>(p.U), *F = static_cast<const __nv_bfloat16 *>(p.F);
            for (int x = first + static_cast<int>(threadIdx.x) - 128; x < last; x += kLfThreads - 128) {
                const int m = x / 128, n = n0 + x % 128;
                const int l = n < p.N ? p.adapters[m] : -1;
                float sum = 0.f;
                if (l >= 0 && l < p.L) {
                    const __nv_bfloat16 *u = U + m * p.ldu, *f = F + (static_cast<int64_t>(l) * p.N + n) * p.ldf;
                    for (int j = 0; j < p.r; j += 64) {
                        uint4 a[8], b[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const bool in = j + 8 * i < p.r;
                            b[i] = in ? *reinterpret_cast<const uint4 *>(f + j + 8 * i) : make_uint4(0, 0, 0, 0);
                            a[i] = in ? __ldcg(reinterpret_cast<const uint4 *>(u + j + 8 * i)) : make_uint4(0, 0, 0, 0);
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            sum = dot8(a[i], b[i], sum);
                    }
                }
                share[x - first] = sum;
            }
        },
        err);
    grid_wait();                     // every warp: no later kernel may start before U's is done
    const __nv_bfloat16 *res = static_cast<const __nv_bfloat16 *>(p.residual);
    __nv_bfloat16 *D = static_cast<__nv_bfloat16 *>(p.D);
    const int64_t limit = (p.M - 1) * p.ldd + p.N;
    const uint32_t part = smem_u32(ring);
    for (int x = first + threadIdx.x; x < last; x += kLfThreads) {
        const int m = x / 128, c = x % 128, n = n0 + c;
        if (n >= p.N)
            continue;
        const float b = p.bias ? p.bias[n] : 0.f, e = res ? __bfloat162float(res[m * p.ld_residual + n]) : 0.f;
        float z = 0.f;
#pragma unroll 8
        for (uint32_t s = 0; s < S; ++s)
            z += ld_cluster_one(part + (m * 128 + c) * 4, s);
        z += share[x - first];
        z += b;
        z += e;
        const int64_t at = m * p.ldd + n;
        if (bounds_ok(at, limit, err, kBndStoreD))
            D[at] = __float2bfloat16_rn(z);
    }
    __syncwarp();
    cluster_sync();                  // no CTA leaves while its partial sums may be read
}

}  // namespace

cudaError_t launch_lora_few_rank(const RankArgs &a, cudaStream_t s)
{
    const int groups = (a.r + kLfRanks - 1) / kLfRanks;
    return launch_overlapped(lora_few_rank_kernel, dim3(static_cast<unsigned>(a.M * groups)), kLfRanks * 32, 0, 1, s, a, groups);
}

cudaError_t launch_lora_few(LoraFewArgs a, int num_sms, const ErrCtx &err, cudaStream_t s)
{
    few_ring(a.shape, kFwRing);
    a.shape.tmem_cols = a.shape.tp <= 32 ? 32 : 64;
    const int64_t tiles = (a.N + 127) / 128;
    const int S = few_cluster(tiles, (a.K + 63) / 64, num_sms);
    const int smem = 1024 + a.shape.ring_bytes + (a.M * 128 / S + 1) * 4;
    const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(lora_few_kernel), smem);
    if (e != cudaSuccess)
        return e;
    return launch_overlapped(lora_few_kernel, dim3(static_cast<unsigned>(tiles * S)), kLfThreads, smem, S, s, a, err);
}

}  // namespace tmg
