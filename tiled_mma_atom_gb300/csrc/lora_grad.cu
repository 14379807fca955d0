// lora_grad.cu — the gradients of the adapters' factors: G[l] = sum over the rows m of
// adapter l of Z[m]^T Y[m], (r, C) or its transpose, on the tensor cores.
//
// Plan.  One block sorts the rows by adapter: a stable counting sort, as the routing's,
// ranking 32 rows at a time per warp with match.any.  It runs beside the kernel that
// makes dU.
//
// Both gradients are one launch: the CTAs of the first side's column tiles, then those
// of the second's.  The contraction over an adapter's rows goes in blocks of 64 of
// them.  A CTA has a tile of 128 columns of Y
// and a run of all adapters' blocks: P runs per tile fill the SMs whatever the
// adapters' shares.  An adapter inside one run is rounded and stored; one that runs
// on leaves fp32 partial sums, which the last of its runs to arrive adds up in
// order, so results do not depend on timing.
//
// Both operands are MN-major (Y's columns on the MMA's M, Z's on its N).  Requests'
// rows are adjacent, so most blocks are 64 rows of Y in a row and come by one box for
// each 64 columns; sixteens of a block that are in a row come by boxes of 16, and
// the others by gathers of four rows, whose numbers past the adapter's last row
// are out of range and read as zeros.  No other adapter's row is ever multiplied: 0
// times its NaN would be NaN.  A row of a box costs the TMA unit about 2.5 ns whatever
// its bytes, so Z's short rows come by cp.async of a warp of their own (by boxes the
// gradients of 8191 x 4096 and 8191 x 4096 took 37 us).
//
// Warps: 0 Y's TMA producer, 1 MMA issuer and TMEM owner, 2..5 epilogue, 6 Z's copies;
// two accumulators in turn.  Bound by HBM: Y once; both gradients of 8191 x 4096 and 8191 x
// 4096, rank 16, 134 MB, 26 us (5.2 TB/s).
#include "feed.cuh"
#include "launch.cuh"
#include "lora.cuh"
#include "lora.h"
#include "pieces.cuh"
#include "staging.cuh"
#include "tc2_kernel.cuh"

namespace tmg {
namespace {

constexpr int kGrThreads = 224;
constexpr int kGrMaxStages = 4;
constexpr int kGrCols = 128;
constexpr int kGrBars = (2 * kGrMaxStages + 4) * 8 + 16;

// The run of a CTA, adapter by adapter.
struct GradWalk {
    const int *unit;
    int L, u, u_end;

    // Adapter, its blocks b0 .. b1 - 1 here, and whether it has others elsewhere.
    __device__ __forceinline__ bool next(int &l, int &b0, int &b1, bool &partial)
    {
        if (u >= u_end)
            return false;
        int lo = 0, hi = L;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (unit[mid] <= u)
                lo = mid;
            else
                hi = mid;
        }
        l = lo;
        const int blocks = unit[l + 1] - unit[l];
        b0 = u - unit[l];
        b1 = min(blocks, b0 + u_end - u);
        partial = b0 != 0 || b1 != blocks;
        u += b1 - b0;
        return true;
    }
};

__device__ __forceinline__ int run_start(int units, int p, int P)
{
    return static_cast<int>(static_cast<int64_t>(units) * p / P);
}

// The runs of a column tile, at most `most`, for the blocks of `some` adapters: sixteen
// blocks each, or as many as the adapters, whose boundaries cost nothing (700 rows of 14
// adapters of rank 32, 1024 x 4096, 45.6 us in one run, 30.1 in seven); but one where the
// blocks and stores that the others take off it are less than ten blocks, what a cut costs
// (700 rows of 2, rank 64, 4096 x 2048, 30.0 us, 37.0 in two).  Grows with blocks and
// adapters, and is never more than the blocks: no run is empty.
__host__ __device__ __forceinline__ int grad_split(int blocks, int some, int most)
{
    const int each = ceil_div(blocks, 16) > some ? ceil_div(blocks, 16) : some, runs = most < each ? most : each;
    return static_cast<int64_t>(blocks + 3 * some) * (runs - 1) <= 10 * runs ? 1 : runs;
}

// Shared memory: wc [32][L], totals [L].
__global__ void __launch_bounds__(1024) lora_plan_kernel(const int32_t *adapters, int M, int L, int32_t *offsets, int32_t *rows)
{
    extern __shared__ int32_t wc[];
    int32_t *total = wc + 32 * L;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    for (int i = threadIdx.x; i < 32 * L; i += 1024)
        wc[i] = 0;
    grid_wait();
    grid_release();
    __syncthreads();
    // each warp's rows are contiguous; four loads of a lane at a time
    const int64_t each = (static_cast<int64_t>(M) + 1023) / 1024 * 32;
    const int64_t m0 = min(static_cast<int64_t>(M), warp * each), m1 = min(static_cast<int64_t>(M), m0 + each);
    int32_t *mine = wc + warp * L;
    auto walk = [&](auto &&with) {
        for (int64_t m = m0; m < m1; m += 128) {
            int l[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t at = m + 32 * i + lane;
                const int x = at < m1 ? adapters[at] : -1;
                l[i] = x < L ? x : -1;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (m + 32 * i >= m1)
                    break;
                with(m + 32 * i + lane, l[i], __match_any_sync(0xffffffffu, l[i]));
                __syncwarp();
            }
        }
    };
    walk([&](int64_t, int l, uint32_t same) {
        if (l >= 0 && lane == __ffs(same) - 1)
            mine[l] += __popc(same);
    });
    __syncthreads();
    for (int l = threadIdx.x; l < L; l += 1024) {
        int sum = 0;
        for (int w = 0; w < 32; ++w)
            sum += wc[w * L + l];
        total[l] = sum;
    }
    __syncthreads();
    if (warp == 0) {
        int run = 0;
        for (int l0 = 0; l0 < L; l0 += 32) {
            const int l = l0 + lane, n = l < L ? total[l] : 0;
            int inc = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o)
                    inc += x;
            }
            if (l < L) {
                total[l] = run + inc - n;
                offsets[l] = run + inc - n;
            }
            run += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0)
            offsets[L] = run;
    }
    __syncthreads();
    for (int l = threadIdx.x; l < L; l += 1024) {
        int at = total[l];
        for (int w = 0; w < 32; ++w) {
            const int n = wc[w * L + l];
            wc[w * L + l] = at;
            at += n;
        }
    }
    __syncthreads();
    walk([&](int64_t m, int l, uint32_t same) {
        const int first = l >= 0 ? mine[l] : 0;
        __syncwarp();
        if (l >= 0) {
            rows[first + __popc(same & ((1u << lane) - 1))] = static_cast<int32_t>(m);
            if (lane == __ffs(same) - 1)
                mine[l] = first + __popc(same);
        }
    });
}

__global__ void __launch_bounds__(kGrThreads) lora_grad_kernel(const __grid_constant__ LoraGradArgs p, ErrCtx err)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + p.stages * p.stage_bytes);
    uint64_t *empty = full + kGrMaxStages;
    uint64_t *tfull = empty + kGrMaxStages;
    uint64_t *tempty = tfull + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(tempty + 2);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *off = reinterpret_cast<int *>(tmem_slot + 4), *unit = off + p.L + 1;

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int tiles0 = ceil_div(p.side[0].C, kGrCols);
    const int which = static_cast<int>(blockIdx.x) >= tiles0 * p.runs ? 1 : 0, cta = blockIdx.x - which * tiles0 * p.runs;
    const LoraGradSide &side = p.side[which];
    const int C = side.C, tiles = ceil_div(C, kGrCols), tile = cta % tiles, run = cta / tiles;
    const int r16 = (p.r + 15) & ~15, acc_cols = (p.r + 31) & ~31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&full[s], 2);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], 4);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane < 3)
        tma_prefetch_desc(&side.tmY[lane]);
    if (warp == 1) {
        tmem_alloc(tmem_slot, p.tmem_cols);
        tmem_relinquish();
    }
    grid_release();
    grid_wait();
    for (int i = threadIdx.x; i <= p.L; i += kGrThreads)
        off[i] = min(max(p.offsets[i], 0), p.M);
    __syncthreads();
    if (warp == 2) {                 // blocks before each adapter
        int sum = 0, some = 0;
        for (int l0 = 0; l0 < p.L; l0 += 32) {
            const int l = l0 + lane;
            const int n = l < p.L ? ceil_div(max(off[l + 1] - off[l], 0), 64) : 0;
            some += __popc(__ballot_sync(0xffffffffu, n > 0));
            int inc = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o)
                    inc += x;
            }
            if (l < p.L)
                unit[l] = sum + inc - n;
            sum += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) {
            unit[p.L] = sum;
            unit[p.L + 1] = grad_split(sum, some, p.runs);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int units = unit[p.L], runs = unit[p.L + 1];
    GradWalk walk{unit, p.L, 0, 0};
    if (run < runs)
        walk = GradWalk{unit, p.L, run_start(units, run, runs), run_start(units, run + 1, runs)};
    int l, b0, b1;
    bool partial;

    if (warp == 0) {
        // ---------------------------------------------- TMA producer
        int stage = 0, issued = 0;
        uint32_t phase = 0;
        bool ok = true;
        while (ok && walk.next(l, b0, b1, partial)) {
            const int end = off[l + 1];
            // lane i: rows i and 32 + i of the next block (past the end: out of range)
            int next[2];
            auto fetch = [&](int b) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int at = off[l] + b * 64 + 32 * h + lane;
                    int m = b < b1 && at < end ? p.rows[at] : -1;
                    next[h] = m < 0 || m >= p.M ? p.M : m;
                }
            };
            fetch(b0);
            for (int b = b0; b < b1; ++b, ++issued) {
                const int m[2] = {next[0], next[1]};
                fetch(b + 1);
                const int left = min(64, end - off[l] - b * 64), sixteens = (left + 15) / 16;
                // which sixteens are rows in a row
                uint32_t whole = 0;
                int first[4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int f = __shfl_sync(0xffffffffu, m[h], lane & 16);
                    const uint32_t in = __ballot_sync(0xffffffffu, m[h] < p.M && m[h] == f + (lane & 15));
                    whole |= ((in & 0xffffu) == 0xffffu ? 1u : 0u) << (2 * h) | (in >> 16 == 0xffffu ? 2u : 0u) << (2 * h);
                    first[2 * h] = __shfl_sync(0xffffffffu, m[h], 0);
                    first[2 * h + 1] = __shfl_sync(0xffffffffu, m[h], 16);
                }
                const bool block = whole == 15 && first[1] == first[0] + 16 && first[2] == first[0] + 32 && first[3] == first[0] + 48;
                if (!mbar_wait_warp(&empty[stage], phase ^ 1u, err, abort_flag, kSiteProducerEmpty)) {
                    ok = false;
                    break;
                }
                mbar_arrive_expect_tx_w(&full[stage], static_cast<uint32_t>(sixteens * 16 * kKBlockBytes * 2));
                uint8_t *sy = smem + stage * p.stage_bytes;
                for (int x = 0; x < 2; ++x) {                     // boxes of 64 columns
                    uint8_t *dst = sy + x * kMnBoxBytes;
                    const CUtensorMap *maps = side.tmY;
                    const int c0 = tile * kGrCols + x * 64;
                    if (block) {
                        tma_load_2d_w(dst, &maps[0], &full[stage], c0, first[0]);
                        continue;
                    }
                    for (int i = 0; i < sixteens; ++i) {
                        uint8_t *to = dst + i * kMnKStepBytes;
                        const int mine = i < 2 ? m[0] : m[1];
                        if (whole >> i & 1) {
                            const int row = i == 0 ? first[0] : i == 1 ? first[1] : i == 2 ? first[2] : first[3];
                            tma_load_2d_w(to, &maps[1], &full[stage], c0, row);
                        } else {
                            const int from = (i & 1) * 16 + (lane & 3) * 4;
                            const int4 four = make_int4(__shfl_sync(0xffffffffu, mine, from), __shfl_sync(0xffffffffu, mine, from + 1),
                                                        __shfl_sync(0xffffffffu, mine, from + 2), __shfl_sync(0xffffffffu, mine, from + 3));
                            if (lane < 4)
                                tma_gather4_one(to + lane * 512, &maps[2], &full[stage], c0, four);
                            __syncwarp();
                        }
                    }
                }
                if (++stage == p.stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        for (int i = 0; i < p.stages && i < issued; ++i) {          // every stage is released
            const int s = stage - 1 - i;
            mbar_wait(&empty[s < 0 ? s + p.stages : s], s < 0 ? phase ^ 1u : phase, err, abort_flag, kSiteDrain);
        }
        if (*abort_flag)
            settle(full, p.stages, stage, phase, min(issued, p.stages), err.word, err.budget_ns);
    } else if (warp == 6) {
        // ------------------------------ Z's rows, as the MMA reads them: 64-rank boxes of
        // rows of 128 bytes, 16-byte chunks swizzled; zeros for rows past the adapter's
        const int chunks = ceil_div(p.r, 8);
        const __nv_bfloat16 *Z = static_cast<const __nv_bfloat16 *>(side.Z);
        int stage = 0, pending = 0, oldest = 0;           // copies under way: stages oldest ..
        uint32_t phase = 0;
        bool ok = true;
        auto land = [&] {                                 // the oldest copies are there: hand them to the MMA
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&full[oldest]);
            oldest = oldest + 1 == p.stages ? 0 : oldest + 1;
            --pending;
        };
        while (ok && walk.next(l, b0, b1, partial)) {
            const int end = off[l + 1];
            int next[2];                                  // lane i: rows i and 32 + i of the next block
            auto fetch = [&](int b) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int at = off[l] + b * 64 + 32 * h + lane;
                    next[h] = b < b1 && at < end ? p.rows[at] : -1;
                }
            };
            fetch(b0);
            for (int b = b0; b < b1; ++b) {
                const int m[2] = {next[0], next[1]};
                fetch(b + 1);
                if (!mbar_wait_warp(&empty[stage], phase ^ 1u, err, abort_flag, kSiteProducerEmpty)) {
                    ok = false;
                    break;
                }
                const uint32_t base = smem_u32(smem + stage * p.stage_bytes) + 2 * kMnBoxBytes + lane * kKBlockBytes;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bool in = m[h] >= 0 && m[h] < p.M;
                    const __nv_bfloat16 *from = Z + (in ? m[h] * side.ldz : 0);
#pragma unroll 4
                    for (int c = 0; c < chunks; ++c)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                         base + (c >> 3) * kMnBoxBytes + 32 * h * kKBlockBytes + (((c & 7) ^ (lane & 7)) << 4)),
                                     "l"(from + c * 8), "r"(in ? 16 : 0)
                                     : "memory");
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                ++pending;
                if (pending == 3) {
                    asm volatile("cp.async.wait_group 2;" ::: "memory");
                    land();
                }
                if (++stage == p.stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        while (pending > 0)
            land();
    } else if (warp == 1) {
        // -------------------------------------------- MMA issuer
        const uint32_t idesc = idesc_bf16_major(kGrCols, r16, 3);
        int stage = 0, local = 0;
        uint32_t phase = 0;
        bool ok = true;
        while (ok && walk.next(l, b0, b1, partial)) {
            const int acc = local & 1, rows = off[l + 1] - off[l];
            const uint32_t acc_phase = (local >> 1) & 1;
            ++local;
            if (!mbar_wait_warp(&tempty[acc], acc_phase ^ 1u, err, abort_flag, kSiteMmaTmemEmpty))
                break;
            tc_fence_after();
            for (int b = b0; b < b1; ++b) {
                if (!mbar_wait_warp(&full[stage], phase, err, abort_flag, kSiteMmaFull)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t y_s = smem_u32(smem + stage * p.stage_bytes);
                const uint64_t ydesc = sdesc_mnmajor_sw128(y_s), zdesc = sdesc_mnmajor_sw128(y_s + 2 * kMnBoxBytes);
                const int steps = (min(64, rows - b * 64) + 15) / 16;
                for (int k = 0; k < steps; ++k)
                    mma_bf16_w(tmem + acc * acc_cols, ydesc + k * (kMnKStepBytes >> 4), zdesc + k * (kMnKStepBytes >> 4), idesc,
                               (b != b0) || (k != 0));
                mma_commit_w(&empty[stage]);
                if (++stage == p.stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok)
                break;
            mma_commit_w(&tfull[acc]);
        }
        if (*abort_flag)
            settle(empty, p.stages, stage, phase, 1, err.word, err.budget_ns);
    } else {
        // ---------------------------------------------------- epilogue
        const int q = warp & 3, col = tile * kGrCols + q * 32 + lane;
        const int64_t limit = static_cast<int64_t>(p.L) * C * p.r;
        __nv_bfloat16 *G = static_cast<__nv_bfloat16 *>(side.G);
        // sixteen ranks from j0 on of this lane's column
        auto store = [&](int adapter, int j0, const float (&v)[16]) {
            if (col >= C)
                return;
            if (side.across) {
                const int64_t at = (static_cast<int64_t>(adapter) * C + col) * p.r + j0;
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (j0 + 8 * h < p.r)
                        store_piece(G, at + 8 * h,
                                    make_uint4(pack_bf16x2(v[8 * h], v[8 * h + 1]), pack_bf16x2(v[8 * h + 2], v[8 * h + 3]),
                                               pack_bf16x2(v[8 * h + 4], v[8 * h + 5]), pack_bf16x2(v[8 * h + 6], v[8 * h + 7])),
                                    min(8, p.r - j0 - 8 * h), limit, err);
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int64_t at = (static_cast<int64_t>(adapter) * p.r + j0 + j) * C + col;
                    if (j0 + j < p.r && bounds_ok(at, limit, err, kBndStoreD))
                        G[at] = __float2bfloat16_rn(v[j]);
                }
            }
        };
        const int64_t piece = static_cast<int64_t>(kGrCols) * r16, p_limit = static_cast<int64_t>(gridDim.x) * 2 * piece;
        // run x's partial sums of adapter a: its first adapter's, or its last's
        auto piece_of = [&](int x, int a) {
            return ((static_cast<int64_t>(which) * tiles0 * p.runs + static_cast<int64_t>(x) * tiles + tile) * 2 + (unit[a] <= run_start(units, x, runs) ? 0 : 1)) * piece + q * 32 + lane;
        };
        int local = 0;
        while (walk.next(l, b0, b1, partial)) {
            const int acc = local & 1;
            const uint32_t acc_phase = (local >> 1) & 1;
            ++local;
            if (!mbar_wait_warp(&tfull[acc], acc_phase, err, abort_flag, kSiteEpiTmemFull))
                break;
            tc_fence_after();
            const int64_t mine = piece_of(run, l);
            for (int j0 = 0; j0 < p.r; j0 += 16) {
                uint32_t t[16];
                tmem_ld16(tmem + (static_cast<uint32_t>(q * 32) << 16) + acc * acc_cols + j0, t);
                float v[16];
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    v[j] = __uint_as_float(t[j]);
                if (!partial) {
                    store(l, j0, v);
                    continue;
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int64_t at = mine + (j0 + j) * kGrCols;
                    if (bounds_ok(at, p_limit, err, kBndPartials))
                        p.partials[at] = v[j];
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&tempty[acc]);
            if (!partial)
                continue;
            const int r_first = unit_owner(unit[l], units, runs), r_last = unit_owner(unit[l + 1] - 1, units, runs);
            const int64_t counter = (static_cast<int64_t>(which) * tiles0 * p.runs + static_cast<int64_t>(r_first) * tiles + tile) * 4 + q;
            if (!last_arrival(p.counters + counter, r_last - r_first, bounds_ok(counter, 4ll * gridDim.x, err, kBndCounters)))
                continue;
            for (int j0 = 0; j0 < p.r; j0 += 16) {
                float v[16] = {};
                for (int x0 = r_first; x0 <= r_last; x0 += 4) {          // four runs' loads in flight
                    float f[4][16];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int64_t at = x0 + x <= r_last ? piece_of(x0 + x, l) + j0 * kGrCols : 0;
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            f[x][j] = x0 + x <= r_last && bounds_ok(at + j * kGrCols, p_limit, err, kBndPartials)
                                          ? __ldcg(p.partials + at + j * kGrCols)
                                          : 0.f;
                    }
#pragma unroll
                    for (int x = 0; x < 4; ++x)
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            v[j] += f[x][j];
                }
                store(l, j0, v);
            }
        }
        // adapters without rows
        const float zeros[16] = {};
        for (int a = run; a < p.L; a += p.runs)
            if (unit[a] == unit[a + 1])
                for (int j0 = 0; j0 < p.r; j0 += 16)
                    store(a, j0, zeros);
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, p.tmem_cols);
    }
}

int64_t grad_tiles(const LoraGradArgs &a)
{
    int64_t n = 0;
    for (int i = 0; i < a.sides; ++i)
        n += (a.side[i].C + kGrCols - 1) / kGrCols;
    return n;
}

// Runs of a column tile, at most: two CTAs per SM.
int grad_runs(const LoraGradArgs &a, int num_sms)
{
    const int64_t fill = 2 * num_sms / grad_tiles(a);
    const int some = a.M < a.L ? a.M : a.L;
    return fill <= 1 ? 1 : grad_split(a.M / 64 + some, some, static_cast<int>(fill));
}

}  // namespace

size_t lora_grad_partial_bytes(const LoraGradArgs &a, int num_sms)
{
    return static_cast<size_t>(grad_runs(a, num_sms)) * grad_tiles(a) * 2 * kGrCols * ((a.r + 15) & ~15) * sizeof(float);
}

int64_t lora_grad_ctas(const LoraGradArgs &a, int num_sms) { return grad_tiles(a) * grad_runs(a, num_sms); }

size_t lora_grad_counters(const LoraGradArgs &a, int num_sms) { return static_cast<size_t>(grad_runs(a, num_sms)) * grad_tiles(a) * 4; }

cudaError_t launch_lora_plan(const int32_t *adapters, int M, int L, int32_t *offsets, int32_t *rows, cudaStream_t s)
{
    const int smem = 33 * L * static_cast<int>(sizeof(int32_t));
    const cudaError_t e = smem > 48 * 1024 ? ensure_smem_attr(reinterpret_cast<const void *>(lora_plan_kernel), smem) : cudaSuccess;
    if (e != cudaSuccess)
        return e;
    return launch_overlapped(lora_plan_kernel, dim3(1), 1024, smem, 1, s, adapters, M, L, offsets, rows);
}

cudaError_t launch_lora_grad(LoraGradArgs a, int num_sms, const ErrCtx &err, cudaStream_t s)
{
    a.runs = grad_runs(a, num_sms);
    a.stage_bytes = (2 + (a.r + 63) / 64) * kMnBoxBytes;
    a.stages = kGrMaxStages;
    a.tmem_cols = 32;
    while (a.tmem_cols < 2 * ((a.r + 31) & ~31))
        a.tmem_cols *= 2;
    const int smem = 1024 + a.stages * a.stage_bytes + kGrBars + 8 * (a.L + 1) + 4;
    const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(lora_grad_kernel), smem);
    if (e != cudaSuccess)
        return e;
    return launch_overlapped(lora_grad_kernel, dim3(static_cast<unsigned>(grad_tiles(a)) * a.runs), kGrThreads, smem, 1, s, a, err);
}

}  // namespace tmg
