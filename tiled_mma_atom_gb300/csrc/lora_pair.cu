// lora_pair.cu — the dense product with low-rank adapters on CTA pairs:
// D[m] = x[m] . W^T + U[m] . F[a_m]^T + bias + residual[m], a tile of 256 rows
// by BN columns per pair as in tc2_kernel.cuh.
//
// The adapters' share is more of the same contraction: after the K blocks of x
// and W come, for every adapter l that a row of the tile has, the blocks of U
// (all 256 rows) and F[l].  Only rows of adapter l may take part, and zeros in the
// others' U would not do: 0 times an infinity in F[l] is NaN in a row that has
// nothing to do with l.  The MMA itself leaves rows out: the accumulator's lanes
// are the rows, and its disable-output-lane operand names the lanes that it does
// not update.  Every warp that needs them finds the tile's adapters from the 256
// row numbers: smallest first (redux), its rows by eight ballots.
//
// Operands.  x, U: boxes of 128 rows.  W and F K-major (the forward product: F[l]
// is (N, r)) or MN-major (the input's gradient: W (contraction, N) and F[l] (r, N) in
// boxes of 64 x 64).  Ranks beyond 64 take several blocks; the columns past r
// are out of range and read as zeros in both operands.
//
// Roles (eleven warps): 0 TMA producer, 1 MMA issuer (CTA 0) and TMEM owner, 2..9
// epilogue, two warps per lane quarter sharing the columns, 10 the tile feed.
// Schedule: swap_kernel.cuh's, tiles taken as pairs get free and the last wave's cut
// along K where that pays.  Cut tiles: the piece with the last K block also takes the
// adapters' blocks.
//
// Bound by the tensor pipe (81 - 84 % busy) like the GEMM's pair kernel: 8191 x 4096 x
// 4096 140 us without adapters, 9 requests of rank 16 add 3; forward 157 - 161 us with the
// ranks, the input's gradient 140.
//
// The kernel that makes U lets this one start as soon as the kernel before it has ended,
// so x, W, F and the row numbers are there; only U's loads wait.  Pairs start as that
// kernel's blocks leave their SMs, up to 10 us apart, which the feed evens out.
#include "feed.cuh"
#include "launch.cuh"
#include "lora.cuh"
#include "lora.h"
#include "pieces.cuh"
#include "staging.cuh"
#include "swap_kernel.cuh"
#include "tc2_kernel.cuh"

namespace tmg {
namespace {

constexpr int kLpThreads = 352;

template <int BN>
struct LoraCfg {
    static constexpr int A_BYTES = kHalfM * kKBlockBytes;
    static constexpr int B_BYTES = (BN / 2) * kKBlockBytes;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int STAGES = 218 * 1024 / STAGE_BYTES > 8 ? 8 : 218 * 1024 / STAGE_BYTES;
    static constexpr int SMEM = 1024 + STAGES * STAGE_BYTES + (2 * STAGES + 4) * 8 + sizeof(FeedSmem) + 16;
};

template <int BN, bool MAJ>
__global__ void __launch_bounds__(kLpThreads, 1) lora_pair_kernel(const __grid_constant__ LoraPairArgs p, ErrCtx err)
{
    using C = LoraCfg<BN>;
    constexpr int STAGES = C::STAGES;
    constexpr uint32_t STAGE_TX = 2u * C::STAGE_BYTES;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    uint8_t *sA = smem, *sB = smem + STAGES * C::A_BYTES;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + STAGES * C::STAGE_BYTES);
    uint64_t *empty = full + STAGES;
    uint64_t *tfull = empty + STAGES;
    uint64_t *tempty = tfull + 2;
    FeedSmem *feed_smem = reinterpret_cast<FeedSmem *>(tempty + 2);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(feed_smem + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = cluster_ctarank();
    const int cluster = blockIdx.x >> 1, nclusters = gridDim.x >> 1;
    const int tiles_m = ceil_div(p.M, kBM), tiles_n = ceil_div(p.N, BN), num_kb = ceil_div(p.K, 64);
    const int rank_blocks = ceil_div(p.r, 64);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], 16);
        }
        feed_init(feed_smem);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane < 4)
        tma_prefetch_desc(lane == 0 ? &p.tmX : lane == 1 ? &p.tmW : lane == 2 ? &p.tmU : &p.tmF);
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, 512);
        tmem_relinquish_pair();
    }
    grid_release();
    tc_fence_before();
    cluster_sync();          // barriers of both CTAs initialised, TMEM allocated
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    const SwapTail tail{p.cut_tiles, p.cut_pieces};
    const int total = tiles_m * tiles_n;
    SwapWalk walk(feed_smem, cluster, nclusters, total, tail, num_kb, err, abort_flag);
    int tile, kb0, kb1, tm, tn;
    bool partial;
    RowAdapters<8> of;

    if (warp == 0) {
        // ---------------------------------------------- TMA producer
        int stage = 0;
        uint32_t phase = 0;
        int64_t issued = 0;
        bool ok = true;
        walk.feed.producer = rank == 0;
        // The next stage of the ring, announced: its place, or -1 where the wait ran out.
        auto take = [&]() -> int {
            if (!mbar_wait_cluster_warp(&empty[stage], phase ^ 1u, err, abort_flag, kSiteProducerEmpty)) {
                ok = false;
                return -1;
            }
            if (rank == 0)
                mbar_arrive_expect_tx_w(&full[stage], STAGE_TX);
            const int at = stage;
            ++issued;
            if (++stage == STAGES) {
                stage = 0;
                phase ^= 1u;
            }
            return at;
        };
        while (ok && walk.next(tile, kb0, kb1, partial)) {
            tile_coords(tile, tiles_m, tiles_n, p.group_m, tm, tn);
            const int a_row = tm * kBM + static_cast<int>(rank) * kHalfM, b_row = tn * BN + static_cast<int>(rank) * (BN / 2);
            if (kb1 == num_kb)
                of.read(p.adapters, static_cast<int64_t>(tm) * kBM, p.M, p.L, lane);
            for (int kb = kb0; kb < kb1; ++kb) {
                const int at = take();
                if (at < 0)
                    break;
                const uint32_t bar0 = mapa_shared(smem_u32(&full[at]), 0);
                tma_load_2d_pair_w(sA + at * C::A_BYTES, &p.tmX, bar0, kb * 64, a_row);
                if constexpr (MAJ) {
#pragma unroll
                    for (int j = 0; j < (BN / 2) / kMnBox; ++j)
                        tma_load_2d_pair_w(sB + at * C::B_BYTES + j * kMnBoxBytes, &p.tmW, bar0, b_row + j * kMnBox, kb * 64);
                } else {
                    tma_load_2d_pair_w(sB + at * C::B_BYTES, &p.tmW, bar0, kb * 64, b_row);
                }
            }
            if (!ok || kb1 != num_kb)
                continue;
            grid_wait();                     // U
            for (int l = of.next(-1); ok && l != kNoAdapter; l = of.next(l))
                for (int c = 0; c < rank_blocks; ++c) {
                    const int at = take();
                    if (at < 0)
                        break;
                    const uint32_t bar0 = mapa_shared(smem_u32(&full[at]), 0);
                    tma_load_2d_pair_w(sA + at * C::A_BYTES, &p.tmU, bar0, c * 64, a_row);
                    if constexpr (MAJ) {
#pragma unroll
                        for (int j = 0; j < (BN / 2) / kMnBox; ++j)
                            tma_load_3d_pair(sB + at * C::B_BYTES + j * kMnBoxBytes, &p.tmF, bar0, b_row + j * kMnBox, c * 64, l);
                    } else {
                        tma_load_3d_pair(sB + at * C::B_BYTES, &p.tmF, bar0, c * 64, b_row, l);
                    }
                }
        }
        // Tail: every stage this CTA filled is released (no multicast arrive still
        // on its way here), and in CTA 0 every load of the pair landed.
        for (int i = 0; i < STAGES && i < issued; ++i) {
            int s = stage - 1 - i;
            uint32_t ph = phase;
            if (s < 0) {
                s += STAGES;
                ph ^= 1u;
            }
            if (rank == 0)
                mbar_wait_cluster(&full[s], ph, err, abort_flag, kSiteDrain);
            mbar_wait_cluster(&empty[s], ph, err, abort_flag, kSiteDrain);
        }
        if (*abort_flag && rank == 0)
            settle(full, STAGES, stage, phase, static_cast<int>(min(issued, static_cast<int64_t>(STAGES))), err.word,
                   err.budget_ns);
    } else if (warp == 1) {
        if (rank == 0) {
            // -------------------------------------------- MMA issuer
            constexpr uint32_t idesc = idesc_bf16_major(kBM, BN, MAJ ? 2 : 0);
            constexpr uint64_t bstep = (MAJ ? kMnKStepBytes : 32) >> 4;
            int stage = 0;
            uint32_t phase = 0;
            int local = 0;
            bool ok = true;
            uint64_t adesc = 0, bdesc = 0;
            auto take = [&] {
                if (!mbar_wait_cluster_warp(&full[stage], phase, err, abort_flag, kSiteMmaFull))
                    return ok = false;
                tc_fence_after();
                const uint32_t b_s = smem_u32(sB + stage * C::B_BYTES);
                adesc = sdesc_kmajor_sw128(smem_u32(sA + stage * C::A_BYTES));
                bdesc = MAJ ? sdesc_mnmajor_sw128(b_s) : sdesc_kmajor_sw128(b_s);
                return true;
            };
            auto give = [&] {
                mma_commit_pair_w(&empty[stage], 0x3);
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            };
            // The next tile is fetched while the last K blocks of this one are under way.
            bool more = walk.next(tile, kb0, kb1, partial);
            while (ok && more) {
                const int acc = local & 1, b0 = kb0, b1 = kb1, turn = max(b0, b1 - 3);
                const uint32_t acc_phase = (local >> 1) & 1;
                ++local;
                tile_coords(tile, tiles_m, tiles_n, p.group_m, tm, tn);
                if (b1 == num_kb)
                    of.read(p.adapters, static_cast<int64_t>(tm) * kBM, p.M, p.L, lane);
                if (!mbar_wait_cluster_warp(&tempty[acc], acc_phase ^ 1u, err, abort_flag, kSiteMmaTmemEmpty))
                    break;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + acc * BN;
                int l = kNoAdapter;                  // the tile's first adapter, found ahead of its turn
                uint32_t off[8];
                for (int kb = b0; kb < b1; ++kb) {
                    if (kb == turn) {
                        if (b1 == num_kb) {
                            l = of.next(-1);
                            of.others(l, off);
                        }
                        more = walk.next(tile, kb0, kb1, partial);
                    }
                    if (!take())
                        break;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_bf16_pair_w(d_tmem, adesc + k * 2, bdesc + k * bstep, idesc, (kb != b0) || (k != 0));
                    give();
                }
                while (ok && l != kNoAdapter) {
                    for (int c = 0; c < rank_blocks && take(); ++c) {
                        const int steps = min(4, ceil_div(p.r - c * 64, 16));
                        for (int k = 0; k < steps; ++k)
                            mma_bf16_pair_masked_w(d_tmem, adesc + k * 2, bdesc + k * bstep, idesc, off);
                        give();
                    }
                    l = of.next(l);
                    of.others(l, off);
                }
                if (!ok)
                    break;
                mma_commit_pair_w(&tfull[acc], 0x3);
            }
            if (*abort_flag)         // the last block's commit (or, before the first, none)
                settle(empty, STAGES, stage, phase, 1, err.word, err.budget_ns);
        }
    } else if (warp == 10) {
        feed_run(feed_smem, rank, total - tail.tiles, nclusters, p.feed, err, abort_flag);
    } else {
        // ---------------------------------------------------- epilogue
        constexpr int CHUNKS = (BN / 32 + 1) / 2;
        const int ew = warp - 2, q = warp & 3;
        const int c_begin = (ew / 4) * CHUNKS, c_end = min(BN / 32, c_begin + CHUNKS);
        const int64_t d_limit = static_cast<int64_t>(p.M - 1) * p.ldd + p.N;
        const int64_t piece = 32 * BN, limit = static_cast<int64_t>(nclusters) * sw_partial_floats(BN);
        __nv_bfloat16 *D = static_cast<__nv_bfloat16 *>(p.D);
        const __nv_bfloat16 *R = static_cast<const __nv_bfloat16 *>(p.residual);
        int local = 0;
        while (walk.next(tile, kb0, kb1, partial)) {
            tile_coords(tile, tiles_m, tiles_n, p.group_m, tm, tn);
            const int acc = local & 1;
            const uint32_t acc_phase = (local >> 1) & 1;
            ++local;
            const int row = tm * kBM + static_cast<int>(rank) * kHalfM + q * 32 + lane;
            // a chunk's residual, read ahead: the next chunk's while one is finished
            uint4 ahead[4];
            const __nv_bfloat16 *res_row = R + static_cast<int64_t>(row) * p.ld_residual;
            auto wide = [&](int c) {
                const int col0 = tn * BN + c * 32;
                return R && c < c_end && row < p.M && col0 + 32 <= p.N && (reinterpret_cast<uintptr_t>(res_row + col0) & 15u) == 0;
            };
            auto read = [&](int c) {
                if (wide(c))
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        ahead[j] = reinterpret_cast<const uint4 *>(res_row + tn * BN + c * 32)[j];
            };
            // bias, residual, rounding and store of a finished chunk
            auto finish = [&](int c, float (&v)[32]) {
                const int col0 = tn * BN + c * 32;
                const bool w = wide(c);
                uint4 here[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    here[j] = ahead[j];
                read(c + 1);
                if (col0 >= p.N)
                    return;
                if (p.bias) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        v[j] += col0 + j < p.N ? p.bias[col0 + j] : 0.f;
                }
                if (row >= p.M)
                    return;
                if (w) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t u4[4] = {here[j].x, here[j].y, here[j].z, here[j].w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            v[8 * j + 2 * i] += __uint_as_float(u4[i] << 16);
                            v[8 * j + 2 * i + 1] += __uint_as_float(u4[i] & 0xffff0000u);
                        }
                    }
                } else if (R) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (col0 + j < p.N)
                            v[j] += __bfloat162float(res_row[col0 + j]);
                }
                const int64_t at = static_cast<int64_t>(row) * p.ldd;
                if (span_ok(at + col0, min(32, p.N - col0), d_limit, err, kBndStoreD))
                    store_row_chunk(D + at, col0, p.N, p.vec_ok, v);
            };
            // The bias's and the residual's loads go through L1, so after this kernel's own
            // wait; the tile's accumulator waits for U's kernel too.
            if (R || p.bias)
                grid_wait();
            if (!partial)
                read(c_begin);
            if (!mbar_wait_cluster(&tfull[acc], acc_phase, err, abort_flag, kSiteEpiTmemFull))
                break;
            tc_fence_after();
            const uint32_t tbase = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * BN;
            const int64_t mine = ((static_cast<int64_t>(cluster) * 2 + rank) * 4 + q) * piece;
#pragma unroll 1
            for (int c = c_begin; c < c_end; ++c) {
                uint32_t t[32];
                tmem_ld32(tbase + c * 32, t);
                float v[32];
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    v[j] = __uint_as_float(t[j]);
                if (!partial) {
                    finish(c, v);
                    continue;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int64_t at = mine + ((c * 8 + j) * 32 + lane) * 4;
                    if (span_ok(at, 4, limit, err, kBndPartials))
                        *reinterpret_cast<float4 *>(p.partials + at) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive_cluster(mapa_shared(smem_u32(&tempty[acc]), 0));
            if (!partial)
                continue;
            const int c_first = tile * walk.each, c_last = c_first + walk.each - 1;
            const int64_t counter = (static_cast<int64_t>(tile) * 2 + rank) * 8 + ew;
            if (!last_arrival(p.counters + counter, c_last - c_first,
                              bounds_ok(counter, static_cast<int64_t>(tail.tiles) * 16, err, kBndCounters)))
                continue;
            read(c_begin);
#pragma unroll 1
            for (int c = c_begin; c < c_end; ++c) {
                float v[32];
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    v[j] = 0.f;
                add_pieces(v, p.partials, limit, c * 1024 + lane * 4, c_first, c_last, [&](int cc) {
                    return ((static_cast<int64_t>(cc) * 2 + rank) * 4 + q) * piece;
                }, err);
                finish(c, v);
            }
        }
    }

    grid_wait();             // every warp: no later kernel may start before U's is done
    __syncwarp();
    tc_fence_before();
    cluster_sync();          // no CTA leaves while its peer may still touch it
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 512);
    }
}

template <int BN, bool MAJ>
cudaError_t launch_lora_as(const LoraPairArgs &a, int pairs, const ErrCtx &err, cudaStream_t s)
{
    using C = LoraCfg<BN>;
    static_assert(C::SMEM <= 232448 && C::STAGES >= 4 && C::B_BYTES % 1024 == 0, "shared memory");
    auto kern = lora_pair_kernel<BN, MAJ>;
    const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(kern), C::SMEM);
    if (e != cudaSuccess)
        return e;
    return launch_overlapped(kern, dim3(static_cast<unsigned>(2 * pairs)), kLpThreads, C::SMEM, 2, s, a, err);
}

}  // namespace

cudaError_t launch_lora_pair(const LoraPairArgs &a, int bn, bool maj, int pairs, const ErrCtx &err, cudaStream_t s)
{
    if (maj)
        return bn == 256 ? launch_lora_as<256, true>(a, pairs, err, s) : launch_lora_as<128, true>(a, pairs, err, s);
    return bn == 256   ? launch_lora_as<256, false>(a, pairs, err, s)
           : bn == 224 ? launch_lora_as<224, false>(a, pairs, err, s)
           : bn == 192 ? launch_lora_as<192, false>(a, pairs, err, s)
                       : launch_lora_as<128, false>(a, pairs, err, s);
}

}  // namespace tmg
