// few.cuh — the product of a few rows with many weights, split over a cluster: 128
// weight rows are the MMA's M, the rows (padded to tp, a multiple of 16) its N, and
// the CTAs of a cluster each sum a run of the tile's K blocks; the partial sums meet
// in shared memory, where every CTA takes a share of the results.
#pragma once

#include "feed.cuh"
#include "launch.cuh"
#include "lora.cuh"

namespace tmg {

constexpr int kFwMaxStages = 12;
constexpr int kFwRing = 96 * 1024;           // bytes that let two CTAs share an SM
constexpr int kFwWeights = 16384;            // 128 weight rows of a K block

struct FewShape {
    int tp;                    // rows rounded up to 16
    int stages, stage_bytes, ring_bytes, tmem_cols;
};

namespace {

struct FewRing {
    uint64_t full[kFwMaxStages], empty[kFwMaxStages], done;
    uint32_t tmem_slot;
    int abort;
    int issued[2];             // stages that the weights' and the rows' producer have issued
};

// sum + the products of eight bf16 with eight others.
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

// Eight consecutive columns of row t of the cluster's S partial tiles.
__device__ __forceinline__ void few_sum(uint32_t part, int t, int col, uint32_t S, float (&z)[8])
{
    cluster_sum8(part + (t * 128 + col) * 4, S, z);
}

__device__ __forceinline__ uint32_t few_cluster_size()
{
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
    return n;
}

// Barriers, TMEM.
__device__ __forceinline__ void few_setup(const FewShape &p, FewRing &sm, const CUtensorMap *weights, const CUtensorMap *rows)
{
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], 1);
        }
        mbar_init(&sm.done, 1);
        sm.abort = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane < 2)
        tma_prefetch_desc(lane ? rows : weights);
    if (warp == 1) {
        tmem_alloc(&sm.tmem_slot, p.tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before();
}

// After a wait ran out and both producers have ended, by one of their warps: the stages that
// settle() has to wait for, the last uses of the ring before the returned number.  Where the
// weights' producer gave up first, the rows' copies of later stages (a ring of them at
// most) are on their way to barriers at which no one arrives any more: announce them.
__device__ __forceinline__ int few_announce(const FewShape &p, FewRing &sm)
{
    int u = sm.issued[0];
    for (; u < sm.issued[1]; ++u)
        mbar_arrive_expect_tx_w(&sm.full[u % p.stages], static_cast<uint32_t>(p.tp) * 128u);
    __syncwarp();
    return u;
}

// The contraction of K blocks kb0 .. kb1 - 1 by warps 0 (weights' producer), 1 (MMA) and
// 2 (rows' producer), then warps 4..7 put the accumulator into the partial tile
// [row][128], over the ring.  load_weights(dst, bar, kb), load_rows(dst, bar, kb): the
// copies of a K block, by a whole warp; wait_rows(): before the first of the rows;
// meanwhile(): what the warps from 4 on do before they wait for the sums.
template <class LoadWeights, class LoadRows, class WaitRows, class Meanwhile>
__device__ __forceinline__ void few_product(const FewShape &p, FewRing &sm, uint8_t *ring, int kb0, int kb1,
                                            LoadWeights &&load_weights, LoadRows &&load_rows, WaitRows &&wait_rows, Meanwhile &&meanwhile,
                                            const ErrCtx &err)
{
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    volatile int *abort_flag = &sm.abort;
    int stage = 0, issued = 0;
    uint32_t phase = 0;
    if (warp == 0 || warp == 2) {
        const uint32_t tx = kFwWeights + static_cast<uint32_t>(p.tp) * 128u;
        if (warp == 2)
            wait_rows();
        for (int kb = kb0; kb < kb1; ++kb, ++issued) {
            if (!mbar_wait_warp(&sm.empty[stage], phase ^ 1u, err, abort_flag, kSiteProducerEmpty))
                break;
            uint8_t *at = ring + stage * p.stage_bytes;
            if (warp == 0) {
                mbar_arrive_expect_tx_w(&sm.full[stage], tx);
                load_weights(at, &sm.full[stage], kb);
            } else {
                load_rows(at + kFwWeights, &sm.full[stage], kb);
            }
            if (++stage == p.stages) {
                stage = 0;
                phase ^= 1u;
            }
        }
        if (lane == 0)
            sm.issued[warp / 2] = issued;
    } else if (warp == 1) {
        const uint32_t idesc = idesc_bf16_f32(128, p.tp);
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!mbar_wait_warp(&sm.full[stage], phase, err, abort_flag, kSiteMmaFull))
                break;
            tc_fence_after();
            const uint32_t w_s = smem_u32(ring + stage * p.stage_bytes);
            const uint64_t wdesc = sdesc_kmajor_sw128(w_s), rdesc = sdesc_kmajor_sw128(w_s + kFwWeights);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                mma_bf16_w(sm.tmem_slot, wdesc + k * 2, rdesc + k * 2, idesc, (kb != kb0) || (k != 0));
            mma_commit_w(&sm.empty[stage]);
            if (++stage == p.stages) {
                stage = 0;
                phase ^= 1u;
            }
        }
        mma_commit_w(&sm.done);
    } else if (warp >= 4) {
        meanwhile();
        if (warp < 8 && mbar_wait_warp(&sm.done, 0, err, abort_flag, kSiteEpiTmemFull)) {
            tc_fence_after();
            const int q = warp & 3;
            const uint32_t part = smem_u32(ring);
            for (int c = 0; c < p.tp; c += 16) {
                uint32_t r[16];
                tmem_ld16(sm.tmem_slot + (static_cast<uint32_t>(q * 32) << 16) + c, r);
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    asm volatile("st.shared.b32 [%0], %1;" ::"r"(part + ((c + j) * 128 + q * 32 + lane) * 4), "r"(kb0 < kb1 ? r[j] : 0u)
                                 : "memory");
            }
            tc_fence_before();
        }
    }
    __syncwarp();
    cluster_sync();                  // every CTA's partial tile is written
    if (warp < 2 && *abort_flag) {
        if (warp == 0) {             // rows and weights share the stages' barriers
            const int n = few_announce(p, sm);
            settle(sm.full, p.stages, n % p.stages, n / p.stages & 1, n, err.word, err.budget_ns);
        } else
            settle(&sm.done, 1, 0, 1, 1, err.word, err.budget_ns);
        __syncwarp();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(sm.tmem_slot, p.tmem_cols);
    }
}

// The ring's stages within `bytes`.
inline void few_ring(FewShape &a, int bytes)
{
    a.stage_bytes = kFwWeights + a.tp * 128;
    a.stages = bytes / a.stage_bytes < kFwMaxStages ? bytes / a.stage_bytes : kFwMaxStages;
    a.ring_bytes = a.stages * a.stage_bytes;
}

// CTAs that share a tile: `ctas` in all at most, four K blocks each at least.
inline int few_cluster(int64_t tiles, int64_t num_kb, int ctas)
{
    int S = 1;
    while (S < 8 && 2 * S * tiles <= ctas && num_kb >= 8 * S)
        S *= 2;
    return S;
}

}  // namespace
}  // namespace tmg
