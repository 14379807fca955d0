// lora_few.cu — the dense product with low-rank adapters for a few rows (decoding): W
// is read once, every row has an adapter of its own.
//
// First kernel: U[m][j], one to eight warps per (row, rank), 16 bytes of X and F per
// lane and load.  Second kernel: W's product as in few.cuh, for which nothing but x is
// needed, so it starts while the first one runs and waits for U only in the eight warps
// that add the adapters' share, whose factors they fetch meanwhile.  The first kernel
// lets the second one start only after its own wait for the kernel before, so x and
// the weights are complete by then.
//
// One kernel for both where the rows have few ranks in all: every cluster makes U again,
// each CTA over the K blocks whose W it streams, beside W's flood.  Up to 32 ranks cost
// 0.1 to 0.6 us on top of the product (1 x 4096 x 4096, rank 16, 9.1 us, in two kernels 10.5;
// 2 x 11000 x 4096 18.1 and 20.0; 1 x 4096 x 1024 6.1 and 5.7), 48 more than the other
// kernel (3 x 4096 x 4096 11.9 and 11.1).
//
// Bound by HBM: W and the rows' factors once.  16 x 8192 x 8192 of rank 16, 139 MB, 27.1
// us (5.1 TB/s, 6.3 while W streams); 1 x 4096 x 4096 9.1 us; 61 rows of rank 64, 32
// adapters, 4096 x 4096 19.5 us.
#include <cuda_bf16.h>

#include "few.cuh"
#include "lora.h"

namespace tmg {
namespace {

constexpr int kLfThreads = 384, kLfWarps = 8;       // warps 4 .. 11 form the adapters' share
constexpr int kLfMaxDepth = 8;
constexpr int kLfManyWarps = 16;             // of the ranks, per SM: two blocks of eight
constexpr int kLfSmem = 108 * 1024;          // of a CTA, where two share an SM
constexpr int kLfBuffer = 4096;              // a warp's room for factors, at least one unit of 32 columns

// J ranks of a row per `parts` warps of the block (a power of two), each with a run
// of C.  Every load of up to 2048 elements a warp is in flight at once, about when the
// next kernel starts: behind its flood of W's blocks they would take 5 us and more.
// Two ranks a warp where there are many: a row's x is read half as often.
template <int J>
__global__ void __launch_bounds__(256, J == 1 ? 3 : 2) lora_few_rank_kernel(RankArgs a, int parts, int groups)
{
    __shared__ float part[8][J];
    grid_wait();
    grid_release();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t unit = blockIdx.x * static_cast<int64_t>(8 / parts) + warp / parts;
    const int64_t m = unit / groups;
    const int j0 = static_cast<int>(unit % groups) * J, p = warp % parts;
    const int l = m < a.M ? a.adapters[m] : -1;
    const bool on = l >= 0 && l < a.L;
    const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.X) + (on ? m * a.ldx : 0));
    const int n = on ? static_cast<int>(a.C / 8) : 0;
    const uint4 *f[J];
#pragma unroll
    for (int j = 0; j < J; ++j)                          // columns past r pad a row: zeros
        f[j] = on && j0 + j < a.r ? reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.F) +
                                                                    (static_cast<int64_t>(l) * a.r + j0 + j) * a.C)
                                  : nullptr;
    float sum[J] = {};
    for (int c = p * 256 + lane; c - lane < n; c += parts * 256) {
        uint4 v[J][8], w[8];
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[j][i] = f[j] && c + 32 * i < n ? f[j][c + 32 * i] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = c + 32 * i < n ? x[c + 32 * i] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sum[j] = dot8(v[j][i], w[i], sum[j]);
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
#pragma unroll
        for (int o = 16; o; o >>= 1)
            sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], o);
        if (lane == 0)
            part[warp][j] = sum[j];
    }
    __syncthreads();
    const int j = j0 + lane;
    if (lane >= J || p != 0 || m >= a.M || (j >= a.r && j >= a.ldu))
        return;
    float u = 0.f;
    for (int i = 0; i < parts; ++i)
        u += part[warp + i][lane];
    if (on && a.scales)
        u *= a.scales[l];
    static_cast<__nv_bfloat16 *>(a.U)[m * a.ldu + j] = __float2bfloat16_rn(j < a.r ? u : 0.f);
}

__device__ __forceinline__ float ld_cluster_one(uint32_t addr, uint32_t rank)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa_shared(addr, rank)) : "memory");
    return v;
}

// Warps 4 .. 11, where U is made here: the rows' ranks, four a warp at most, over this
// CTA's K blocks.  The sums go to every CTA of the cluster, part[CTA][rank].
__device__ __forceinline__ void send_ranks(const LoraFewArgs &p, float (*part)[kLoraFewWith], uint64_t *bar, int kb0, int kb1, uint32_t S,
                                           uint32_t rank)
{
    constexpr int n = kLoraFewWith / kLfWarps;
    const int warp = threadIdx.x / 32 - 4, lane = threadIdx.x % 32, units = p.M * p.r;
    const int lo = kb0 * 8, hi = min(kb1 * 64, p.K) / 8;       // in 16 bytes
    const uint4 *f[n], *x[n];
    float sum[n];
#pragma unroll
    for (int i = 0; i < n; ++i) {
        const int unit = warp + i * kLfWarps, m = unit / p.r, j = unit - m * p.r;
        const int l = unit < units ? p.adapters[m] : -1;
        sum[i] = 0.f;
        x[i] = f[i] = nullptr;
        if (l >= 0 && l < p.L) {
            x[i] = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.X) + m * p.ldx);
            f[i] = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.A) + (static_cast<int64_t>(l) * p.r + j) * p.K);
        }
    }
    for (int c = lo + lane; c - lane < hi; c += 64) {
        uint4 v[n][2], w[n][2];
#pragma unroll
        for (int i = 0; i < n; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bool in = f[i] && c + 32 * h < hi;
                v[i][h] = in ? f[i][c + 32 * h] : make_uint4(0, 0, 0, 0);
                w[i][h] = in ? x[i][c + 32 * h] : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
        for (int i = 0; i < n; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                sum[i] = dot8(v[i][h], w[i][h], sum[i]);
    }
#pragma unroll
    for (int i = 0; i < n; ++i) {
        const int unit = warp + i * kLfWarps;
        if (unit >= units)
            break;
#pragma unroll
        for (int o = 16; o; o >>= 1)
            sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
        if (lane < static_cast<int>(S))
            st_async_u32(mapa_shared(smem_u32(&part[rank][unit]), lane), __float_as_uint(sum[i]), mapa_shared(smem_u32(bar), lane));
        __syncwarp();
    }
}

// Warps 4 .. 11.  The results of this CTA in units of 32 columns of a row, a warp's
// in turn: their factor rows, 32 x ldf contiguous elements, come by bulk copies, as
// many units ahead as the warp's room holds and the first ones before U is there.
// share[] = U[m] . F[a_m][n] + bias + residual.  A lane takes the 16-byte chunks of
// its factor row from a start of its own, so that eight lanes touch all banks.
// get_ranks(m0, rows): those rows' U to us[row][ldu], by all eight warps.
template <class GetRanks>
__device__ __forceinline__ void adapters_share(const LoraFewArgs &p, uint8_t *room, uint64_t *bars, __nv_bfloat16 *us, float *share,
                                               int n0, int first, int last, GetRanks &&get_ranks, volatile int *abort_flag,
                                               const ErrCtx &err)
{
    const int warp = threadIdx.x / 32 - 4, lane = threadIdx.x % 32;
    const int unit_bytes = static_cast<int>(32 * p.ldf * 2), depth = p.room_bytes / unit_bytes, chunks = static_cast<int>(p.ldf / 8);
    const __nv_bfloat16 *F = static_cast<const __nv_bfloat16 *>(p.F);
    const __nv_bfloat16 *res = static_cast<const __nv_bfloat16 *>(p.residual);
    uint32_t pending = 0;                                // slots with a copy under way
    // copy unit x's factor rows (of columns inside N) if its row has an adapter, l
    auto fetch = [&](int x, int slot, int l) {
        const int n = n0 + x % 4 * 32;
        if (n >= p.N || l < 0 || l >= p.L)
            return;
        pending |= 1u << slot;
        const uint32_t bytes = static_cast<uint32_t>(min(32, p.N - n)) * static_cast<uint32_t>(p.ldf * 2);
        mbar_arrive_expect_tx_w(&bars[slot], bytes);
        bulk_load_w(room + slot * unit_bytes, F + (static_cast<int64_t>(l) * p.N + n) * p.ldf, bytes, &bars[slot]);
    };
    for (int d = 0; d < depth && first + warp + d * kLfWarps < last; ++d) {
        const int x = first + warp + d * kLfWarps;
        fetch(x, d, __ldcg(p.adapters + x / 4));         // before the wait: past L1
    }
    const int m0 = first / 4, rows = last > first ? (last - 1) / 4 - m0 + 1 : 0;
    const int per = static_cast<int>(p.ldu / 8);
    get_ranks(m0, rows);
    asm volatile("bar.sync 1, 256;" ::: "memory");
    uint32_t phases = 0;                                 // of the slots
    int slot = 0;
    for (int x = first + warp; x < last; x += kLfWarps) {
        const int m = x / 4, n = n0 + x % 4 * 32 + lane, l = p.adapters[m];
        float sum = 0.f, add = 0.f;
        if (n < p.N) {
            add = p.bias ? p.bias[n] : 0.f;
            if (res)
                add += __bfloat162float(res[m * p.ld_residual + n]);
        }
        if (l >= 0 && l < p.L && n - lane < p.N) {
            if (!mbar_wait_warp(&bars[slot], phases >> slot & 1u, err, abort_flag, kSiteMmaFull)) {
                for (int d = 0; d < depth; ++d)          // leave when the copies have landed
                    if (pending >> d & 1u)
                        settle(&bars[d], 1, 0, phases >> d & 1u ? 0u : 1u, 1, err.word, err.budget_ns);
                return;
            }
            phases ^= 1u << slot;
            pending &= ~(1u << slot);
            const uint4 *f = reinterpret_cast<const uint4 *>(room + slot * unit_bytes) + lane * chunks;
            const uint4 *u = reinterpret_cast<const uint4 *>(us) + (m - m0) * per;
            int k = (lane * chunks >> 3) % chunks;
            if (n < p.N)
                for (int i = 0; i < chunks; ++i) {
                    sum = dot8(u[k], f[k], sum);
                    k = k + 1 == chunks ? 0 : k + 1;
                }
        }
        share[(x - first) * 32 + lane] = sum + add;
        __syncwarp();
        if (x + depth * kLfWarps < last)
            fetch(x + depth * kLfWarps, slot, p.adapters[(x + depth * kLfWarps) / 4]);
        slot = slot + 1 == depth ? 0 : slot + 1;
    }
}

// WITH: U is made here too.
template <bool WITH>
__global__ void __launch_bounds__(kLfThreads, 2) lora_few_kernel(const __grid_constant__ LoraFewArgs p, ErrCtx err)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ FewRing sm;
    __shared__ uint64_t bars[kLfWarps][kLfMaxDepth];
    __shared__ uint64_t ranks_bar;
    __shared__ float ranks_part[WITH ? 8 : 1][kLoraFewWith];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t *ring = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    uint8_t *room = ring + p.shape.ring_bytes;
    __nv_bfloat16 *us = reinterpret_cast<__nv_bfloat16 *>(room + kLfWarps * p.room_bytes);
    const uint32_t rank = cluster_ctarank(), S = few_cluster_size();
    const int n0 = blockIdx.x / S * 128, num_kb = ceil_div(p.K, 64), warp = threadIdx.x / 32;
    const int kb0 = static_cast<int>(static_cast<int64_t>(num_kb) * rank / S);
    const int kb1 = static_cast<int>(static_cast<int64_t>(num_kb) * (rank + 1) / S);
    // this CTA's results: units of 32 columns of a row
    const int units = p.M * 4, first = units * rank / S, last = units * (rank + 1) / S;
    float *share = reinterpret_cast<float *>(us + (ceil_div(last - first, 4) + 1) * p.ldu);
    if (threadIdx.x < kLfWarps * kLfMaxDepth)
        mbar_init(&bars[0][0] + threadIdx.x, 1);
    few_setup(p.shape, sm, &p.tmW, &p.tmX);
    if (WITH && threadIdx.x == 0) {
        mbar_init(&ranks_bar, 1);
        mbar_arrive_expect_tx(&ranks_bar, S * static_cast<uint32_t>(p.M * p.r) * 4u);
    }
    __syncwarp();
    fence_mbar_init();
    grid_release();
    if constexpr (WITH) {
        cluster_sync();              // the barriers that the others' sums arrive at
        grid_wait();
    } else {
        __syncthreads();
    }
    tc_fence_after();
    auto get_ranks = [&](int m0, int rows) {
        const int thread = threadIdx.x - 128;
        if constexpr (WITH) {
            send_ranks(p, ranks_part, &ranks_bar, kb0, kb1, S, rank);
            if (!mbar_wait_cluster_warp(&ranks_bar, 0, err, &sm.abort, kSiteMmaFull))
                settle(&ranks_bar, 1, 0, 1, 1, err.word, err.budget_ns);
            auto sum = [&](int m, int j) {
                const int l = p.adapters[m];
                float u = 0.f;
                if (j < p.r && l >= 0 && l < p.L) {
                    for (uint32_t x = 0; x < S; ++x)
                        u += ranks_part[x][m * p.r + j];
                    if (p.scales)
                        u *= p.scales[l];
                }
                return __float2bfloat16_rn(u);
            };
            const int ldu = static_cast<int>(p.ldu);
            for (int i = thread; i < rows * ldu; i += kLfWarps * 32)
                us[i] = sum(m0 + i / ldu, i % ldu);
            if (p.U && blockIdx.x == 0)
                for (int i = thread; i < p.M * p.r; i += kLfWarps * 32)
                    static_cast<__nv_bfloat16 *>(p.U)[i] = sum(i / p.r, i % p.r);
        } else {
            grid_wait();
            const int per = static_cast<int>(p.ldu / 8);
            for (int i = thread; i < rows * per; i += kLfWarps * 32)
                reinterpret_cast<uint4 *>(us)[i] =
                    __ldcg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.U) + (m0 + i / per) * p.ldu) + i % per);
        }
    };
    few_product(
        p.shape, sm, ring, kb0, kb1, [&](uint8_t *dst, uint64_t *bar, int kb) { tma_load_2d_w(dst, &p.tmW, bar, kb * 64, n0); },
        [&](uint8_t *dst, uint64_t *bar, int kb) { tma_load_2d_w(dst, &p.tmX, bar, kb * 64, 0); }, [] {},
        [&] {
            adapters_share(p, room + (warp - 4) * p.room_bytes, bars[warp - 4], us, share, n0, first, last, get_ranks, &sm.abort,
                           err);
        },
        err);
    if (!WITH)
        grid_wait();                 // every warp: no later kernel may start before U's is done
    __nv_bfloat16 *D = static_cast<__nv_bfloat16 *>(p.D);
    const int64_t limit = (p.M - 1) * p.ldd + p.N;
    const uint32_t part = smem_u32(ring);
    for (int x = first * 32 + threadIdx.x; x < last * 32; x += kLfThreads) {
        const int m = x / 128, c = x % 128, n = n0 + c;
        if (n >= p.N)
            continue;
        float z = 0.f;
#pragma unroll 8
        for (uint32_t s = 0; s < S; ++s)
            z += ld_cluster_one(part + (m * 128 + c) * 4, s);
        z += share[x - first * 32];
        const int64_t at = m * p.ldd + n;
        if (bounds_ok(at, limit, err, kBndStoreD))
            D[at] = __float2bfloat16_rn(z);
    }
    __syncwarp();
    cluster_sync();                  // no CTA leaves while its partial sums may be read
}

}  // namespace

cudaError_t launch_lora_few_rank(const RankArgs &a, int num_sms, cudaStream_t s)
{
    int parts = 1;
    while (parts < 8 && a.C > 2048 * parts)
        parts *= 2;
    const int ranks = static_cast<int>(a.ldu > a.r && a.ldu < a.r + 8 ? a.ldu : a.r);
    const int J = a.M * ranks * parts > int64_t{kLfManyWarps} * num_sms ? 2 : 1, groups = (ranks + J - 1) / J;
    const int64_t blocks = (a.M * groups + 8 / parts - 1) / (8 / parts);
    return launch_overlapped(J == 1 ? lora_few_rank_kernel<1> : lora_few_rank_kernel<2>, dim3(static_cast<unsigned>(blocks)), 256, 0,
                             1, s, a, parts, groups);
}

// Where a cluster reads few ranks beside the weights of its 128 columns, and is one:
// st.async, by which the sums travel, needs a launch in clusters.
bool lora_few_with(int64_t M, int64_t N, int64_t K, int64_t r, int num_sms)
{
    return N > 0 && K > 0 && M * r <= kLoraFewWith && few_cluster((N + 127) / 128, (K + 63) / 64, 2 * num_sms) > 1;
}

cudaError_t launch_lora_few(LoraFewArgs a, int num_sms, const ErrCtx &err, cudaStream_t s)
{
    const int64_t tiles = (a.N + 127) / 128;
    const int unit = static_cast<int>(32 * a.ldf * 2);
    a.room_bytes = unit >= kLfBuffer ? unit : kLfBuffer / unit > kLfMaxDepth ? kLfMaxDepth * unit : kLfBuffer / unit * unit;
    a.shape.tmem_cols = a.shape.tp <= 32 ? 32 : 64;
    int S = 1, rest = 0;
    for (int per_sm = 2; per_sm >= 1; --per_sm) {      // two CTAs per SM where two stages fit so, else one
        S = few_cluster(tiles, (a.K + 63) / 64, per_sm * num_sms);
        const int units = (a.M * 4 + S - 1) / S;       // of a CTA, at most
        rest = kLfWarps * a.room_bytes + ((units + 3) / 4 + 1) * static_cast<int>(a.ldu) * 2 + units * 128;
        few_ring(a.shape, 2 / per_sm * kLfSmem - rest);
        if (a.shape.stages >= 2)
            break;
    }
    if (a.shape.stages < 2 || (a.A && S < 2))
        return cudaErrorInvalidValue;                  // more ranks than kLoraFewRanks; not lora_few_with()
    const int smem = 1024 + a.shape.ring_bytes + rest;
    auto kern = a.A ? lora_few_kernel<true> : lora_few_kernel<false>;
    const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(kern), smem);
    if (e != cudaSuccess)
        return e;
    return launch_overlapped(kern, dim3(static_cast<unsigned>(tiles * S)), kLfThreads, smem, S, s, a, err);
}

}  // namespace tmg
