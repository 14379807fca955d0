// lora_rank.cu — U[m] = bf16(scales[a_m] X[m] . F[a_m]^T) on the tensor cores: the
// low-rank side of the products with adapters for many rows.
//
// A tile is 128 rows of X; a cluster of S CTAs (1, 2, 4 or 8) shares it, each CTA
// taking a run of its K blocks, and the fp32 partial sums meet in shared memory as in
// split_kernel.cuh.  A K block of X is loaded once and multiplied with the same
// block of each adapter that a row of the tile has; the accumulator's lanes are
// the rows, and an MMA leaves those of other adapters out (disable-output-lane), so
// one accumulator of r columns is enough, and what another adapter holds, infinities
// too, reaches no row that is not its own.  An adapter's first MMA writes, the later
// ones add, so nothing needs clearing; rows without an adapter are written as zeros.
// A stage holds the blocks of `chunk` adapters; where a tile has more, it goes
// over X again for the next ones.
//
// F K-major, (L, r, C), or MN-major, (L, C, r), in boxes of 64 x 64 whose columns past
// r read as zeros.  Warps: 0 TMA producer, 1 MMA issuer and TMEM owner, 2..5 the
// rows' scales and the accumulator's way to shared memory; all six add up the partials.
//
// Bound by HBM: X once.  8191 x 4096, rank 16: 12 - 15 us (4.5 - 5.6 TB/s); 700 x 4096, rank
// 32: 7 us, latency.
#include "feed.cuh"
#include "launch.cuh"
#include "lora.cuh"
#include "lora.h"
#include "staging.cuh"
#include "tc2_kernel.cuh"

namespace tmg {
namespace {

constexpr int kRkThreads = 192;
constexpr int kRkRows = 128;
constexpr int kRkMaxStages = 8;
constexpr int kRkChunk = 8192;          // a stage's room for adapters' blocks, one at least
constexpr int kRkBars = (2 * kRkMaxStages + 1) * 8 + 24;      // barriers; TMEM address, abort flag, number of adapters
constexpr int kRkLists = kRkRows * (16 + 4 + 8);              // masks and numbers of the tile's adapters; rows' scales and whether they have one

template <bool MAJ>
__global__ void __launch_bounds__(kRkThreads) lora_rank_kernel(const __grid_constant__ LoraRankArgs p, ErrCtx err)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    uint4 *masks = reinterpret_cast<uint4 *>(smem + p.ring_bytes);
    int *list = reinterpret_cast<int *>(masks + kRkRows);
    float *scale = reinterpret_cast<float *>(list + kRkRows);
    int *has = reinterpret_cast<int *>(scale + kRkRows);
    uint64_t *full = reinterpret_cast<uint64_t *>(has + kRkRows);
    uint64_t *empty = full + kRkMaxStages;
    uint64_t *done = empty + kRkMaxStages;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *count = reinterpret_cast<int *>(tmem_slot + 2);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int S = p.cluster;
    const uint32_t rank = cluster_ctarank();
    const int row0 = blockIdx.x / S * kRkRows, num_kb = ceil_div(p.C, 64);
    const int kb0 = static_cast<int>(static_cast<int64_t>(num_kb) * rank / S);
    const int kb1 = static_cast<int>(static_cast<int64_t>(num_kb) * (rank + 1) / S);

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(done, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane < 2)
        tma_prefetch_desc(lane ? &p.tmF : &p.tmX);
    if (warp == 1) {
        tmem_alloc(tmem_slot, p.tmem_cols);
        tmem_relinquish();
    }
    if (!p.beside)
        grid_wait();
    grid_release();                  // only now: the product reads x without a wait
    if (warp == 0) {
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
    const int n = *count;
    const uint32_t part = smem_u32(smem), width = ((p.r + 15) & ~15) + 4;      // the partial sums [row][width], over the ring

    int stage = 0, issued = 0;
    uint32_t phase = 0;
    if (warp == 0) {
        // ---------------------------------------------- TMA producer
        for (int first = 0; first < n && !*abort_flag; first += p.chunk) {
            const int here = min(p.chunk, n - first);
            for (int kb = kb0; kb < kb1; ++kb, ++issued) {
                if (!mbar_wait_warp(&empty[stage], phase ^ 1u, err, abort_flag, kSiteProducerEmpty))
                    break;
                uint8_t *sx = smem + stage * p.stage_bytes, *sf = sx + kRkRows * kKBlockBytes;
                mbar_arrive_expect_tx_w(&full[stage], kRkRows * kKBlockBytes + here * p.block_bytes);
                tma_load_2d_w(sx, &p.tmX, &full[stage], kb * 64, row0);
                for (int i = 0; i < here; ++i, sf += p.block_bytes) {
                    const int l = list[first + i];
                    if constexpr (MAJ) {
                        for (int j = 0; j * 64 < p.r; ++j)
                            tma_load_3d_one(sf + j * kMnBoxBytes, &p.tmF, &full[stage], j * 64, kb * 64, l);
                    } else {
                        tma_load_3d_one(sf, &p.tmF, &full[stage], kb * 64, 0, l);
                    }
                }
                if (++stage == p.stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
    } else if (warp == 1) {
        // -------------------------------------------- MMA issuer
        const uint32_t idesc = idesc_bf16_major(kRkRows, (p.r + 15) & ~15, MAJ ? 2 : 0);
        constexpr uint64_t fstep = (MAJ ? kMnKStepBytes : 32) >> 4;
        for (int first = 0; first < n && !*abort_flag; first += p.chunk) {
            const int here = min(p.chunk, n - first);
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!mbar_wait_warp(&full[stage], phase, err, abort_flag, kSiteMmaFull))
                    break;
                tc_fence_after();
                const uint32_t x_s = smem_u32(smem + stage * p.stage_bytes), f_s = x_s + kRkRows * kKBlockBytes;
                const uint64_t xdesc = sdesc_kmajor_sw128(x_s);
                for (int i = 0; i < here; ++i) {
                    const uint4 off = masks[first + i];
                    const uint32_t at = f_s + i * p.block_bytes;
                    const uint64_t fdesc = MAJ ? sdesc_mnmajor_sw128(at) : sdesc_kmajor_sw128(at);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_bf16_masked_w(tmem, xdesc + k * 2, fdesc + k * fstep, idesc, off, (kb != kb0) || (k != 0));
                }
                mma_commit_w(&empty[stage]);
                if (++stage == p.stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        mma_commit_w(done);
    } else {
        const int q = warp & 3, row = q * 32 + lane;
        const int64_t m = static_cast<int64_t>(row0) + row;
        const int l = m < p.M ? __ldcg(p.adapters + m) : -1;         // `beside`: before this kernel's wait
        has[row] = l >= 0 && l < p.L;
        scale[row] = has[row] && p.scales ? __ldcg(p.scales + l) : 1.f;
        if (mbar_wait_warp(done, 0, err, abort_flag, kSiteEpiTmemFull)) {
            // --------------------- the accumulator to shared memory
            tc_fence_after();
            for (int c = 0; c < p.r; c += 16) {
                uint32_t t[16];
                tmem_ld16(tmem + (static_cast<uint32_t>(q * 32) << 16) + c, t);
#pragma unroll
                for (int j = 0; j < 16; j += 4)
                    sts128(part + (row * width + c + j) * 4, kb0 < kb1 ? make_uint4(t[j], t[j + 1], t[j + 2], t[j + 3]) : make_uint4(0, 0, 0, 0));
            }
            tc_fence_before();
        }
    }
    __syncwarp();
    cluster_sync();                  // every CTA's partial sums are written
    if (warp < 2 && *abort_flag) {
        if (warp == 0)
            settle(full, p.stages, stage, phase, issued, err.word, err.budget_ns);
        else
            settle(done, 1, 0, 1, 1, err.word, err.budget_ns);
        __syncwarp();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, p.tmem_cols);
    }
    // ------------------------- this CTA's share of the rows, eight ranks at a time
    __nv_bfloat16 *U = static_cast<__nv_bfloat16 *>(p.U);
    const int64_t limit = p.M * p.ldu;
    const int share = kRkRows / S, groups = ceil_div(p.r, 8);
    for (int i = threadIdx.x; i < share * groups; i += kRkThreads) {
        const int row = static_cast<int>(rank) * share + i / groups, j0 = i % groups * 8;
        const int64_t m = static_cast<int64_t>(row0) + row;
        if (m >= p.M)
            continue;
        float v[8];
        cluster_sum8(part + (row * width + j0) * 4, S, v);
#pragma unroll
        for (int j = 0; j < 8; ++j)              // zeros without an adapter, and in the columns that pad a row
            v[j] = has[row] && j0 + j < p.r ? v[j] * scale[row] : 0.f;
        store_piece(U, m * p.ldu + j0,
                    make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])),
                    static_cast<int>(min(static_cast<int64_t>(8), p.ldu - j0)), limit, err);
    }
    if (p.beside)
        grid_wait();                 // what comes after this kernel comes after the one before it
    __syncwarp();
    cluster_sync();                  // no CTA leaves while its partial sums may be read
}

}  // namespace

cudaError_t launch_lora_rank_tc(LoraRankArgs a, bool maj, int num_sms, const ErrCtx &err, cudaStream_t s)
{
    const int tiles = (a.M + kRkRows - 1) / kRkRows, num_kb = (a.C + 63) / 64, r16 = (a.r + 15) & ~15;
    // Two CTAs per SM where the ring allows it, at least four K blocks each.
    a.cluster = 1;
    while (a.cluster < 8 && 2ll * a.cluster * tiles <= 2 * num_sms && num_kb >= 8 * a.cluster)
        a.cluster *= 2;
    a.block_bytes = maj ? (a.r + 63) / 64 * kMnBoxBytes : r16 * kKBlockBytes;
    // The ring: half an SM's shared memory, or more where few CTAs run.
    const int few = 2 * tiles * a.cluster <= num_sms, ring = few ? 196608 : 98304, room = few ? 2 * kRkChunk : kRkChunk;
    a.chunk = a.block_bytes >= room ? 1 : room / a.block_bytes;
    a.stage_bytes = kRkRows * kKBlockBytes + a.chunk * a.block_bytes;
    a.stages = ring / a.stage_bytes < 2 ? 2 : ring / a.stage_bytes > kRkMaxStages ? kRkMaxStages : ring / a.stage_bytes;
    a.ring_bytes = a.stages * a.stage_bytes;
    if (a.ring_bytes < (r16 + 4) * kRkRows * 4)
        a.ring_bytes = (r16 + 4) * kRkRows * 4;
    a.tmem_cols = 32;
    while (a.tmem_cols < r16)
        a.tmem_cols *= 2;
    auto kern = maj ? lora_rank_kernel<true> : lora_rank_kernel<false>;
    const int smem = 1024 + a.ring_bytes + kRkLists + kRkBars;
    const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(kern), smem);
    if (e != cudaSuccess)
        return e;
    return launch_overlapped(kern, dim3(static_cast<unsigned>(tiles) * a.cluster), kRkThreads, smem, a.cluster, s, a, err);
}

}  // namespace tmg
