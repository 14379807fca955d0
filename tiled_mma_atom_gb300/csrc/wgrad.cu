// wgrad.cu — the weight gradient of the expert-grouped product on CTA pairs:
// dB[e] (N, K) = dD_eᵀ · A_e, the contraction over the rows of group e.
//
// Both operands are stored with the contraction as their outer dimension, so
// both are MN-major MMA operands: 64 x 64 boxes (64 rows of 128 bytes, 128-byte
// swizzle).  A pair tile is 256 columns of dD by 256 (at the edge: 128) columns
// of A.  A block of the contraction is 64 rows of the group.
//
// Groups end anywhere.  Rows past the end belong to the next group and may hold
// NaN or infinities, so zeroing one operand is not enough: the last block of a
// group is read in pieces up to the next multiple of 16 rows (one MMA step):
// boxes of 16 rows while they lie inside the group, and for the rest TMA
// gathers of four rows each whose indices past the end are out of range and
// read as zeros (issued by a warp of their own: 16 gathers take 0.7 us, which
// the producer would lose on the next tile).  The MMA steps beyond are not
// issued.  Rows by number are gathered into workspace before this kernel.  A
// group without rows is one such block of zeros: its tile is written as zeros
// like any other.
//
// Schedule: every group has the same tiles (bands of `group` column tiles), of
// as many blocks as the group has; pairs take them as they get free (feed.cuh).
// Where few tiles would be left for the last wave, as many of the first are cut
// over 2 to 8 pairs each and summed from fp32 partials in pair order.  Roles as in swap_kernel.cuh.
//
// Results leave by TMA from swizzled 4 KB tiles, a warp's 32 rows of 64 columns,
// where dB has 16-byte rows (128 groups of 16 rows, 2048 x 1024, 537 MB of dB: 97
// us, 5.5 TB/s, against 124 with stores of each lane).
//
// Bound by the tensor pipe (65 % busy) and, in short groups, by the epilogue:
// 65528 rows over 64 groups, 2048 x 1024, 185 us (1.49 PFLOP/s).
#include "feed.cuh"
#include "grouped.h"
#include "launch.cuh"
#include "pieces.cuh"
#include "staging.cuh"
#include "tc2_kernel.cuh"
#include "wgrad.h"

namespace tmg {
namespace {

constexpr int kWgMaxStages = 6;
constexpr int kWgStaging = 8 * 4096;             // a warp's 32 rows of 64 columns
constexpr int kWgStageBytes = 32768;
constexpr int kWgBars = (3 * kWgMaxStages + 4) * 8 + sizeof(FeedSmem) + 16;  // barriers, feed, TMEM address, abort flag
constexpr int64_t kWgPiece = 32 * 256;
constexpr int kWgThreads = 384;                  // producer, MMA, eight epilogue warps, feed, group ends

__host__ inline int wg_smem(int stages, int E)
{
    return 1024 + stages * kWgStageBytes + kWgStaging + kWgBars + 8 * (E + 1);
}

__device__ __forceinline__ void tma_gather4_pair_to(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, const int4 &r)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes.cta_group::2"
                 " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w)
                 : "memory");
}

// The warp's staging tile (32 rows of 128 bytes, swizzled) to dB; rows and columns
// outside are left out.
__device__ __forceinline__ void tma_store_tile(const CUtensorMap *map, uint32_t src, int col, int row, int e)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];\n\t"
                 "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(map)), "r"(col), "r"(row), "r"(e), "r"(src)
                 : "memory");
}

// Blocks of a group's contraction (one of zeros for an empty group).
__device__ __forceinline__ int wg_blocks(int rows) { return rows > 0 ? ceil_div(rows, 64) : 1; }

// The walk of a pair: its run of split blocks first, then whole tiles.
struct WgWalk {
    const int *off, *unit;        // group offsets; blocks before each group
    Feed feed;
    int per, E, sk;
    int64_t u, u_end;
    bool first;
    const ErrCtx &err;
    volatile int *abort;

    __device__ WgWalk(FeedSmem *f, int c, int nc, int sk_, int64_t U, int cut, int total, int per_, int E_, const int *off_,
                      const int *unit_, const ErrCtx &er, volatile int *ab)
        : off(off_), unit(unit_), feed(f, c, nc, total - sk_), per(per_), E(E_), sk(sk_), u(c < cut ? U * c / cut : 0),
          u_end(c < cut ? U * (c + 1) / cut : 0), first(true), err(er), abort(ab)
    {
    }

    __device__ int rows(int e) const { return max(off[e + 1] - off[e], 0); }

    __device__ bool next(int &e, int &local, int &kb0, int &kb1, bool &partial, int &slot, int64_t &unit0, int &blocks)
    {
        if (u < u_end) {
            int lo = 0, hi = E;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (unit[mid] <= u)
                    lo = mid;
                else
                    hi = mid;
            }
            e = lo;
            blocks = wg_blocks(rows(e));
            const int64_t in = u - unit[e];
            local = static_cast<int>(in / blocks);
            unit0 = unit[e] + static_cast<int64_t>(local) * blocks;
            kb0 = static_cast<int>(u - unit0);
            kb1 = static_cast<int>(min(static_cast<int64_t>(blocks), kb0 + (u_end - u)));
            partial = kb0 != 0 || kb1 != blocks;
            slot = first ? 0 : 1;
            first = false;
            u += kb1 - kb0;
            return true;
        }
        int tile;
        if (!feed.next(tile, err, abort))
            return false;
        e = (tile + sk) / per;
        local = (tile + sk) % per;
        blocks = wg_blocks(rows(e));
        kb0 = 0;
        kb1 = blocks;
        partial = false;
        slot = 0;
        unit0 = 0;
        return true;
    }
};

__global__ void __launch_bounds__(kWgThreads, 1) wgrad_kernel(const __grid_constant__ WgradTmaArgs p, ErrCtx err)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    uint8_t *staging = smem + p.stages * kWgStageBytes;
    uint64_t *full = reinterpret_cast<uint64_t *>(staging + kWgStaging);
    uint64_t *empty = full + kWgMaxStages;
    uint64_t *tfull = empty + kWgMaxStages;
    uint64_t *tempty = tfull + 2;
    uint64_t *go = tempty + 2;                   // the producer has set up a stage with a group's end
    FeedSmem *feed_smem = reinterpret_cast<FeedSmem *>(go + kWgMaxStages);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(feed_smem + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *off = reinterpret_cast<int *>(tmem_slot + 4), *unit = off + p.E + 1;

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = cluster_ctarank();
    const int cluster = blockIdx.x >> 1, nclusters = gridDim.x >> 1;
    const int tiles_n = ceil_div(p.N, 256), tiles_k = ceil_div(p.K, 256), per = tiles_n * tiles_k;

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
            mbar_init(&go[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], 16);
        }
        feed_init(feed_smem, kFeedReaders + 2);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane < 6)
        tma_prefetch_desc(lane == 0   ? &p.tmA
                          : lane == 1 ? &p.tmD
                          : lane == 2 ? &p.tmA16
                          : lane == 3 ? &p.tmD16
                          : lane == 4 ? &p.tmAg
                                      : &p.tmDg);
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, 512);
        tmem_relinquish_pair();
    }
    grid_release();
    grid_wait();
    for (int i = threadIdx.x; i <= p.E; i += kWgThreads)
        off[i] = p.offsets ? min(max(p.offsets[i], 0), p.R) : (i ? p.R : 0);
    __syncthreads();
    if (warp == 2) {                 // blocks before each group
        int run = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + lane;
            const int n = e < p.E ? wg_blocks(off[e + 1] - off[e]) * per : 0;
            int inc = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o)
                    inc += x;
            }
            if (e < p.E)
                unit[e] = run + inc - n;
            run += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0)
            unit[p.E] = run;
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    const int total = p.E * per, rem = total % nclusters;
    int sk = 0, cut = 0;             // split tiles, pairs that share their blocks
    int64_t U = 0;
    const int each = rem ? min(8, nclusters / rem) : 0;
    if (p.partials && each >= 2) {
        const int e = rem / per, blocks = e < p.E ? wg_blocks(off[e + 1] - off[e]) : 0;
        const int64_t units = unit[e] + static_cast<int64_t>(rem % per) * blocks;
        // a tile's blocks, on average, less a piece's, against what a cut costs
        // in blocks (6.5 us + 0.6 a piece)
        if (unit[p.E] / total * (each - 1) > (kWgCutBlocks + 2 * each) * each && units >= rem * each) {
            sk = rem;
            cut = rem * each;
            U = units;
        }
    }
    WgWalk walk(feed_smem, cluster, nclusters, sk, U, cut, total, per, p.E, off, unit, err, abort_flag);
    int e, local_tile, kb0, kb1, slot, blocks, tn, tk;
    int64_t unit0;
    bool partial;

    if (warp == 0) {
        // ---------------------------------------------- TMA producer
        int stage = 0;
        uint32_t phase = 0;
        int64_t issued = 0;
        bool ok = true;
        walk.feed.producer = rank == 0;
        while (ok && walk.next(e, local_tile, kb0, kb1, partial, slot, unit0, blocks)) {
            tile_coords(local_tile, tiles_n, tiles_k, p.group, tn, tk);
            const int lo = off[e], hi = lo + walk.rows(e);
            const int kcols = p.K - tk * 256 <= 128 ? 64 : 128;               // columns of A per CTA
            const int n0 = tn * 256 + static_cast<int>(rank) * 128, k0 = tk * 256 + static_cast<int>(rank) * kcols;
            const int abox = kcols / 64;
            for (int kb = kb0; kb < kb1; ++kb) {
                const int r0 = lo + kb * 64, left = hi - r0;
                const bool whole = left >= 64;
                const int rows16 = whole ? 64 : (max(left, 1) + 15) & ~15;
                if (!mbar_wait_cluster_warp(&empty[stage], phase ^ 1u, err, abort_flag, kSiteProducerEmpty)) {
                    ok = false;
                    break;
                }
                if (rank == 0)
                    mbar_arrive_expect_tx_w(&full[stage], 2u * static_cast<uint32_t>((2 + abox) * rows16 * 128));
                const uint32_t bar0 = mapa_shared(smem_u32(&full[stage]), 0);
                uint8_t *sd = smem + stage * kWgStageBytes, *sa = sd + 16384;
                if (whole) {
                    tma_load_2d_pair_w(sd, &p.tmD, bar0, n0, r0);
                    tma_load_2d_pair_w(sd + kMnBoxBytes, &p.tmD, bar0, n0 + kMnBox, r0);
                    tma_load_2d_pair_w(sa, &p.tmA, bar0, k0, r0);
                    if (abox == 2)
                        tma_load_2d_pair_w(sa + kMnBoxBytes, &p.tmA, bar0, k0 + kMnBox, r0);
                } else {
                    for (int i = 0; i + 16 <= left; i += 16) {
                        tma_load_2d_pair_w(sd + i * 128, &p.tmD16, bar0, n0, r0 + i);
                        tma_load_2d_pair_w(sd + kMnBoxBytes + i * 128, &p.tmD16, bar0, n0 + kMnBox, r0 + i);
                        tma_load_2d_pair_w(sa + i * 128, &p.tmA16, bar0, k0, r0 + i);
                        if (abox == 2)
                            tma_load_2d_pair_w(sa + kMnBoxBytes + i * 128, &p.tmA16, bar0, k0 + kMnBox, r0 + i);
                    }
                    if (lane == 0 && (left <= 0 || (left & 15)))
                        mbar_arrive(&go[stage]);       // the last, partial sixteen: warp 11
                }
                ++issued;
                if (++stage == p.stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        for (int i = 0; i < p.stages && i < issued; ++i) {
            int s = stage - 1 - i;
            uint32_t ph = phase;
            if (s < 0) {
                s += p.stages;
                ph ^= 1u;
            }
            if (rank == 0)
                mbar_wait_cluster(&full[s], ph, err, abort_flag, kSiteDrain);
            mbar_wait_cluster(&empty[s], ph, err, abort_flag, kSiteDrain);
        }
        if (*abort_flag && rank == 0)
            settle(full, p.stages, stage, phase, static_cast<int>(min(issued, static_cast<int64_t>(p.stages))), err.word,
                   err.budget_ns);
    } else if (warp == 1) {
        if (rank == 0) {
            // -------------------------------------------- MMA issuer
            int stage = 0;
            uint32_t phase = 0;
            int count = 0;
            bool ok = true;
            while (ok && walk.next(e, local_tile, kb0, kb1, partial, slot, unit0, blocks)) {
                tile_coords(local_tile, tiles_n, tiles_k, p.group, tn, tk);
                const int rows = walk.rows(e);
                const uint32_t idesc = idesc_bf16_major(256, p.K - tk * 256 <= 128 ? 128 : 256, 3);
                const int acc = count & 1;
                const uint32_t acc_phase = (count >> 1) & 1;
                ++count;
                if (!mbar_wait_cluster_warp(&tempty[acc], acc_phase ^ 1u, err, abort_flag, kSiteMmaTmemEmpty))
                    break;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + acc * 256;
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!mbar_wait_cluster_warp(&full[stage], phase, err, abort_flag, kSiteMmaFull)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t s0 = smem_u32(smem + stage * kWgStageBytes);
                    const uint64_t adesc = sdesc_mnmajor_sw128(s0), bdesc = sdesc_mnmajor_sw128(s0 + 16384);
                    const int steps = min(4, (max(rows - kb * 64, 1) + 15) / 16);
                    for (int k = 0; k < steps; ++k)
                        mma_bf16_pair_w(d_tmem, adesc + k * (kMnKStepBytes >> 4), bdesc + k * (kMnKStepBytes >> 4), idesc,
                                        (kb != kb0) || (k != 0));
                    mma_commit_pair_w(&empty[stage], 0x3);
                    if (++stage == p.stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok)
                    break;
                mma_commit_pair_w(&tfull[acc], 0x3);
            }
            if (*abort_flag)         // the last K block's commit (or, before the first, none)
                settle(empty, p.stages, stage, phase, 1, err.word, err.budget_ns);
        }
    } else if (warp == 11) {
        // ------------------- gathers of the last, partial sixteen rows of a group
        int stage = 0;
        uint32_t phases = 0;             // one bit per stage
        while (walk.next(e, local_tile, kb0, kb1, partial, slot, unit0, blocks)) {
            const int r0 = off[e] + (blocks - 1) * 64, left = walk.rows(e) - (blocks - 1) * 64;
            const int at = (stage + kb1 - kb0 - 1) % p.stages;
            stage = (stage + kb1 - kb0) % p.stages;
            if (kb1 != blocks || (left > 0 && !(left & 15)))
                continue;
            if (!mbar_wait_warp(&go[at], (phases >> at) & 1u, err, abort_flag, kSiteProducerEmpty))
                break;
            phases ^= 1u << at;
            tile_coords(local_tile, tiles_n, tiles_k, p.group, tn, tk);
            const int kcols = p.K - tk * 256 <= 128 ? 64 : 128;
            const int n0 = tn * 256 + static_cast<int>(rank) * 128, k0 = tk * 256 + static_cast<int>(rank) * kcols;
            // lane 4 b + g: rows 4 g .. 4 g + 3 of the sixteen, box b of dD
            // (0, 1) or A (2, 3)
            const int in = ((max(left, 1) + 15) & ~15) - 16 + 4 * (lane & 3), b = lane >> 2;
            if (b < 2 + kcols / 64) {
                int4 r;
                r.x = in + 0 < left ? r0 + in + 0 : p.R;
                r.y = in + 1 < left ? r0 + in + 1 : p.R;
                r.z = in + 2 < left ? r0 + in + 2 : p.R;
                r.w = in + 3 < left ? r0 + in + 3 : p.R;
                const uint32_t sd = smem_u32(smem + at * kWgStageBytes) + (b < 2 ? 0 : 16384);
                tma_gather4_pair_to(sd + (b & 1) * kMnBoxBytes + in * 128, b < 2 ? &p.tmDg : &p.tmAg,
                                    mapa_shared(smem_u32(&full[at]), 0), (b < 2 ? n0 : k0) + (b & 1) * kMnBox, r);
            }
            __syncwarp();
        }
    } else if (warp == 10) {
        feed_run(feed_smem, rank, total - sk, nclusters, p.feed, err, abort_flag);
    } else {
        // ---------------------------------------------------- epilogue
        const int ew = warp - 2, half = ew / 4, q = warp & 3;
        int count = 0;
        const int64_t d_limit = static_cast<int64_t>(p.E) * p.N * p.K;
        const int64_t p_limit = nclusters * 16 * kWgPiece;
        while (walk.next(e, local_tile, kb0, kb1, partial, slot, unit0, blocks)) {
            tile_coords(local_tile, tiles_n, tiles_k, p.group, tn, tk);
            const int acc = count & 1;
            const uint32_t acc_phase = (count >> 1) & 1;
            ++count;
            const int width = p.K - tk * 256 <= 128 ? 128 : 256;
            const int n = tn * 256 + static_cast<int>(rank) * 128 + q * 32 + lane;
            if (!mbar_wait_cluster(&tfull[acc], acc_phase, err, abort_flag, kSiteEpiTmemFull))
                break;
            tc_fence_after();
            const uint32_t tbase = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * 256;
            const int c1 = min(width / 32, (p.K - tk * 256 + 31) / 32);       // 32-column chunks with columns
            const int pairs = (c1 + 1) / 2;                                   // of which the warp takes every other two
            bool finish = !partial;
            int c_first = 0, c_last = 0;
            if (partial) {
                const int64_t mine = ((static_cast<int64_t>(2 * cluster + slot) * 2 + rank) * 4 + q) * kWgPiece;
#pragma unroll 1
                for (int c = 2 * half; c < c1; c += (c & 1) ? 3 : 1) {
                    uint32_t r[32];
                    tmem_ld32(tbase + c * 32, r);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int64_t at = mine + ((c * 8 + j) * 32 + lane) * 4;
                        if (span_ok(at, 4, p_limit, err, kBndPartials))
                            *reinterpret_cast<uint4 *>(p.partials + at) =
                                make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_cluster(mapa_shared(smem_u32(&tempty[acc]), 0));
                if (half < pairs) {
                    c_first = unit_owner(unit0, U, cut);
                    c_last = unit_owner(unit0 + blocks - 1, U, cut);
                    const int64_t at = ((static_cast<int64_t>(e) * per + local_tile) * 2 + rank) * 8 + ew;
                    finish = last_arrival(p.counters + at, c_last - c_first,
                                          bounds_ok(at, 2ll * nclusters * 16, err, kBndCounters));
                }
            }
            if (finish) {
                __nv_bfloat16 *D = static_cast<__nv_bfloat16 *>(p.dB);
                const int64_t first = static_cast<int64_t>(e) * p.N * p.K;
                const int n0 = n - lane;
                const uint32_t stg = smem_u32(staging + ew * 4096);
#pragma unroll 1
                for (int pr = half; pr < pairs; pr += 2) {
                    if (p.tma_out) {
                        if (lane == 0)                          // the tile's last store has read it
                            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                        __syncwarp();
                    }
                    // this lane's row, 64 columns, to the staging tile in
                    // 16-byte pieces (swizzled)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int c = 2 * pr + h;
                        float v[32];
                        if (!partial) {
                            uint32_t r[32];
                            tmem_ld32(tbase + c * 32, r);
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                v[j] = __uint_as_float(r[j]);
                        } else {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                v[j] = 0.f;
                            if (c < c1)
                                add_pieces(v, p.partials, p_limit, c * 1024 + lane * 4, c_first, c_last, [&](int cc) {
                                    const int s2 = U * cc / cut >= unit0 ? 0 : 1;   // its run begins in this tile
                                    return ((static_cast<int64_t>(2 * cc + s2) * 2 + rank) * 4 + q) * kWgPiece;
                                }, err);
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            sts128(stg + lane * 128 + (((4 * h + j) ^ (lane & 7)) << 4),
                                   make_uint4(pack_bf16x2(v[8 * j], v[8 * j + 1]), pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                                              pack_bf16x2(v[8 * j + 4], v[8 * j + 5]), pack_bf16x2(v[8 * j + 6], v[8 * j + 7])));
                    }
                    if (p.tma_out) {
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                        if (lane == 0 && n0 < p.N)
                            tma_store_tile(&p.tmOut, stg, tk * 256 + pr * 64, n0, e);
                        continue;
                    }
                    __syncwarp();
                    // whole 128-byte lines out: eight lanes a row
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int row = 4 * i + (lane >> 3), piece = lane & 7, col = tk * 256 + pr * 64 + piece * 8;
                        const uint4 v = lds128(stg + row * 128 + ((piece ^ (row & 7)) << 4));
                        if (n0 + row >= p.N || col >= p.K)
                            continue;
                        store_piece(D, first + static_cast<int64_t>(n0 + row) * p.K + col, v, min(8, p.K - col), d_limit, err);
                    }
                    __syncwarp();
                }
            }
            if (!partial) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_cluster(mapa_shared(smem_u32(&tempty[acc]), 0));
            }
        }
        if (p.tma_out && lane == 0)
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }

    __syncwarp();
    tc_fence_before();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 512);
    }
}

}  // namespace

size_t wgrad_partial_bytes(int num_sms) { return static_cast<size_t>(num_sms / 2) * 16 * kWgPiece * sizeof(float); }

cudaError_t launch_wgrad(const WgradTmaArgs &a, int num_sms, const ErrCtx &err, cudaStream_t s)
{
    WgradTmaArgs p = a;
    p.stages = kWgMaxStages;
    while (wg_smem(p.stages, p.E) > 232448)
        --p.stages;
    const int smem = wg_smem(p.stages, p.E);
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(wgrad_kernel), smem);
    if (e != cudaSuccess)
        return e;
    return launch_overlapped(wgrad_kernel, dim3(2 * (num_sms / 2)), kWgThreads, smem, 2, s, p, err);
}

}  // namespace tmg
