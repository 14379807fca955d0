// lora_split.cu — the dense product with low-rank adapters where there are too few
// tiles for the CTA pairs: a tile of 128 rows by 128 columns per CTA, shared by a
// cluster of S CTAs (1, 2, 4 or 8) that each sum a run of its K blocks and of its
// adapters' blocks.
//
// As in lora_pair.cu the accumulator's lanes are the rows, and an MMA on an adapter's
// block leaves out the rows of others.  The fp32 partial sums meet in shared memory as
// in split_kernel.cuh, in rank order; each CTA finishes a share of the rows.
// Only U's loads wait for the kernel that makes it.
//
// Warps: 0 TMA producer, 1 MMA issuer and TMEM owner, 4..7 the accumulator's way to
// shared memory; all eight add up the partial sums.
//
// Bound by latency: 700 x 1024 x 4096, rank 32, 48 tiles over clusters of two, 16 us, of
// them 9 for x and W beside the ranks, 2 for the adapters' blocks, 4 for the sums.
#include "feed.cuh"
#include "launch.cuh"
#include "lora.cuh"
#include "lora.h"
#include "staging.cuh"
#include "tc2_kernel.cuh"

namespace tmg {
namespace {

constexpr int kLsThreads = 256;
constexpr int kLsMinStages = 3, kLsMaxStages = 5;
constexpr int kLsStageBytes = 32768;
constexpr int kLsTile = 128;
constexpr int kLsBars = (2 * kLsMaxStages + 1) * 8 + 24;    // barriers; TMEM address, abort flag, number of adapters
constexpr int kLsWidth = kLsTile + 4;                       // of a row of partial sums
static_assert(kLsTile * kLsWidth * 4 <= kLsMinStages * kLsStageBytes, "the partial sums lie over the ring");

template <bool MAJ>
__global__ void __launch_bounds__(kLsThreads) lora_split_kernel(const __grid_constant__ LoraPairArgs p, int S, int stages, ErrCtx err)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    uint4 *masks = reinterpret_cast<uint4 *>(smem + stages * kLsStageBytes);
    int *list = reinterpret_cast<int *>(masks + kLsTile);
    uint64_t *full = reinterpret_cast<uint64_t *>(list + kLsTile);
    uint64_t *empty = full + kLsMaxStages;
    uint64_t *done = empty + kLsMaxStages;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *count = reinterpret_cast<int *>(tmem_slot + 2);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = cluster_ctarank();
    const int tiles_m = ceil_div(p.M, kLsTile), num_kb = ceil_div(p.K, 64), rank_blocks = ceil_div(p.r, 64);
    const int tile = blockIdx.x / S, row0 = tile % tiles_m * kLsTile, col0 = tile / tiles_m * kLsTile;
    const int kb0 = static_cast<int>(static_cast<int64_t>(num_kb) * rank / S);
    const int kb1 = static_cast<int>(static_cast<int64_t>(num_kb) * (rank + 1) / S);

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(done, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane < 4)
        tma_prefetch_desc(lane == 0 ? &p.tmX : lane == 1 ? &p.tmW : lane == 2 ? &p.tmU : &p.tmF);
    if (warp == 1) {
        tmem_alloc(tmem_slot, kLsTile);
        tmem_relinquish();
    }
    grid_release();
    if (warp == 4) {
        // the tile's adapters, smallest first, and the lanes that each leaves out
        RowAdapters<4> of;
        of.read(p.adapters, row0, p.M, p.L, lane);
        int n = 0;
        for (int l = of.next(-1); l != kNoAdapter; l = of.next(l), ++n) {
            uint32_t off[4];
            of.others(l, off);
            if (lane == 0) {
                masks[n] = make_uint4(off[0], off[1], off[2], off[3]);
                list[n] = l;
            }
        }
        if (lane == 0)
            *count = n;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // this CTA's adapters' blocks
    const int extra = *count * rank_blocks, x0 = extra * static_cast<int>(rank) / S, x1 = extra * (static_cast<int>(rank) + 1) / S;

    int stage = 0, issued = 0;
    uint32_t phase = 0;
    if (warp == 0) {
        // ---------------------------------------------- TMA producer
        bool ok = true;
        auto take = [&] {
            if (!mbar_wait_warp(&empty[stage], phase ^ 1u, err, abort_flag, kSiteProducerEmpty))
                return ok = false;
            mbar_arrive_expect_tx_w(&full[stage], kLsStageBytes);
            return true;
        };
        auto step = [&] {
            ++issued;
            if (++stage == stages) {
                stage = 0;
                phase ^= 1u;
            }
        };
        for (int kb = kb0; kb < kb1 && take(); ++kb, step()) {
            uint8_t *sx = smem + stage * kLsStageBytes, *sw = sx + kLsStageBytes / 2;
            tma_load_2d_w(sx, &p.tmX, &full[stage], kb * 64, row0);
            if constexpr (MAJ) {
                tma_load_2d_w(sw, &p.tmW, &full[stage], col0, kb * 64);
                tma_load_2d_w(sw + kMnBoxBytes, &p.tmW, &full[stage], col0 + kMnBox, kb * 64);
            } else {
                tma_load_2d_w(sw, &p.tmW, &full[stage], kb * 64, col0);
            }
        }
        if (x0 < x1)
            grid_wait();                     // U
        for (int x = x0; ok && x < x1 && take(); ++x, step()) {
            uint8_t *sx = smem + stage * kLsStageBytes, *sw = sx + kLsStageBytes / 2;
            const int l = list[x / rank_blocks], c = x % rank_blocks * 64;
            tma_load_2d_w(sx, &p.tmU, &full[stage], c, row0);
            if constexpr (MAJ) {
                tma_load_3d_one(sw, &p.tmF, &full[stage], col0, c, l);
                tma_load_3d_one(sw + kMnBoxBytes, &p.tmF, &full[stage], col0 + kMnBox, c, l);
            } else {
                tma_load_3d_one(sw, &p.tmF, &full[stage], c, col0, l);
            }
        }
    } else if (warp == 1) {
        // -------------------------------------------- MMA issuer
        constexpr uint32_t idesc = idesc_bf16_major(kLsTile, kLsTile, MAJ ? 2 : 0);
        constexpr uint64_t wstep = (MAJ ? kMnKStepBytes : 32) >> 4;
        bool ok = true;
        uint64_t xdesc = 0, wdesc = 0;
        auto take = [&] {
            if (!mbar_wait_warp(&full[stage], phase, err, abort_flag, kSiteMmaFull))
                return ok = false;
            tc_fence_after();
            const uint32_t x_s = smem_u32(smem + stage * kLsStageBytes), w_s = x_s + kLsStageBytes / 2;
            xdesc = sdesc_kmajor_sw128(x_s);
            wdesc = MAJ ? sdesc_mnmajor_sw128(w_s) : sdesc_kmajor_sw128(w_s);
            return true;
        };
        auto give = [&] {
            mma_commit_w(&empty[stage]);
            if (++stage == stages) {
                stage = 0;
                phase ^= 1u;
            }
        };
        for (int kb = kb0; kb < kb1 && take(); ++kb) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                mma_bf16_w(tmem, xdesc + k * 2, wdesc + k * wstep, idesc, (kb != kb0) || (k != 0));
            give();
        }
        for (int x = x0; ok && x < x1 && take(); ++x) {
            const uint4 off = masks[x / rank_blocks];
            const int steps = min(4, ceil_div(p.r - x % rank_blocks * 64, 16));
            for (int k = 0; k < steps; ++k)
                mma_bf16_masked_w(tmem, xdesc + k * 2, wdesc + k * wstep, idesc, off, 1u);
            give();
        }
        mma_commit_w(done);
    } else if (warp >= 4 && mbar_wait_warp(done, 0, err, abort_flag, kSiteEpiTmemFull)) {
        // ------------------------- the accumulator to shared memory
        tc_fence_after();
        const int q = warp & 3;
        const uint32_t at = smem_u32(smem) + (q * 32 + lane) * kLsWidth * 4;
        for (int c = 0; c < kLsTile; c += 32) {
            uint32_t t[32];
            tmem_ld32(tmem + (static_cast<uint32_t>(q * 32) << 16) + c, t);
#pragma unroll
            for (int j = 0; j < 32; j += 4)
                sts128(at + (c + j) * 4, make_uint4(t[j], t[j + 1], t[j + 2], t[j + 3]));
        }
        tc_fence_before();
    }
    __syncwarp();
    cluster_sync();                  // every CTA's partial sums are written
    if (warp < 2 && *abort_flag) {
        if (warp == 0)
            settle(full, stages, stage, phase, issued, err.word, err.budget_ns);
        else
            settle(done, 1, 0, 1, 1, err.word, err.budget_ns);
        __syncwarp();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kLsTile);
    }
    grid_wait();                     // every warp: no later kernel may start before U's is done
    // ------------------------- this CTA's share of the rows, eight columns at a time
    __nv_bfloat16 *D = static_cast<__nv_bfloat16 *>(p.D);
    const __nv_bfloat16 *R = static_cast<const __nv_bfloat16 *>(p.residual);
    const int64_t limit = (p.M - 1) * p.ldd + p.N;
    const int share = kLsTile / S;
    const uint32_t part = smem_u32(smem);
    for (int i = threadIdx.x; i < share * (kLsTile / 8); i += kLsThreads) {
        const int row = static_cast<int>(rank) * share + i / (kLsTile / 8), c = i % (kLsTile / 8) * 8, col = col0 + c, n = min(8, p.N - col);
        const int64_t m = static_cast<int64_t>(row0) + row;
        if (m >= p.M || n <= 0)
            continue;
        float e[8] = {};
        if (R) {
            const __nv_bfloat16 *r = R + m * p.ld_residual + col;
            if (n == 8 && (reinterpret_cast<uintptr_t>(r) & 15u) == 0) {
                const uint4 v = *reinterpret_cast<const uint4 *>(r);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    e[2 * j] = __uint_as_float(w[j] << 16);
                    e[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    e[j] = j < n ? __bfloat162float(r[j]) : 0.f;
            }
        }
        float z[8];
        cluster_sum8(part + (row * kLsWidth + c) * 4, S, z);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            z[j] += (p.bias && j < n ? p.bias[col + j] : 0.f) + e[j];
        store_piece(D, m * p.ldd + col,
                    make_uint4(pack_bf16x2(z[0], z[1]), pack_bf16x2(z[2], z[3]), pack_bf16x2(z[4], z[5]), pack_bf16x2(z[6], z[7])),
                    n, limit, err);
    }
    __syncwarp();
    cluster_sync();                  // no CTA leaves while its partial sums may be read
}

}  // namespace

cudaError_t launch_lora_split(const LoraPairArgs &a, bool maj, int cluster, const ErrCtx &err, cudaStream_t s)
{
    auto kern = maj ? lora_split_kernel<true> : lora_split_kernel<false>;
    // One CTA per SM and a deep ring (700 x 1024 x 4096 19.0 -> 16.0 us, 128 x 8192 x 8192
    // 37.7 -> 33.5), but two for clusters of eight, of which too few find eight free SMs
    // otherwise (500 x 512 x 8192 23.1 us, 28.8 deep), and for gradients, whose next kernel
    // starts on the SMs beside this one (100 x 4096 x 4096 34.8 us, 37.7 deep; 128 x 8192 x
    // 8192 57.7, 54.5 deep).
    const int stages = (maj || cluster > 4) ? kLsMinStages : kLsMaxStages;
    const int smem = 1024 + stages * kLsStageBytes + kLsTile * 20 + kLsBars;
    const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(kern), smem);
    if (e != cudaSuccess)
        return e;
    const int64_t tiles = static_cast<int64_t>((a.M + kLsTile - 1) / kLsTile) * ((a.N + kLsTile - 1) / kLsTile);
    return launch_overlapped(kern, dim3(static_cast<unsigned>(tiles * cluster)), kLsThreads, smem, cluster, s, a, cluster, stages, err);
}

}  // namespace tmg
