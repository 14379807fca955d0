// split_kernel.cuh — the grouped and the dense product where there are too few
// tiles for the SMs (few rows, narrow matrices): Dᵀ = B · Aᵀ as in
// swap_kernel.cuh, but a tile is 128 weight rows of one CTA, and a cluster of S
// CTAs (1, 2, 4 or 8) shares one tile, each CTA summing a run of its K blocks.
//
// The sums meet in shared memory: every CTA leaves its fp32 partial tile in its
// own (where the operand ring was), and after one cluster barrier each takes a
// share of the tile's rows of A, adds the S partials in rank order (so results
// do not depend on timing) and runs the epilogue on them, eight output columns
// per thread.  A split through global memory costs a pair 6 us and more
// (partials, fence, counter, partials back); this one 0.8 us at 16 rows and 2.7 at
// 128.  At 16 x 4096 x 4096 with the weights in L2 the product took 16.8 us with
// the pair kernel and takes 8.6 so.
//
// Operands are the pair kernel's: weights K-major or MN-major through 3-D maps
// (SwiGLU: 64 gate rows and their 64 up rows, two boxes), A by boxes of the
// tile's width or TMA gathers of named rows.  Warps: 0 the weights' TMA producer,
// 1 MMA issuer and TMEM owner, 2..9 epilogue, 2 before that the rows' producer;
// all ten add up the partials.
//
// Bound by HBM where the weights do not come from L2: one token's 8 experts, 67
// MB, 17.1 us; 16 x 8192 x 8192, 134 MB, 24.7.  A kernel that only reads takes
// 14.7 us for 63 MB and 24.6 for 126.
#pragma once

#include "act.cuh"
#include "feed.cuh"
#include "grouped.h"
#include "launch.cuh"
#include "split.h"
#include "staging.cuh"
#include "swap_kernel.cuh"

namespace tmg {
namespace {

constexpr int kSplitThreads = 320;
constexpr int kSplitBars = (2 * kSplitMaxStages + 2) * 8 + 16 + 1024;   // barriers, TMEM address, abort flag, row numbers
static_assert((kSplitBars - 1024) % 16 == 0, "the row numbers are read in 16-byte pieces");

__device__ __forceinline__ void tma_load_3d_w(void *dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1, int c2)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];\n\t}" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap *map, uint64_t *bar, int c0, const int4 &r)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w)
                 : "memory");
}

__device__ __forceinline__ void mma_e4m3_w(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
    return n;
}

// Four floats of the partial tile of CTA `rank` of the cluster.
__device__ __forceinline__ float4 ld_partial(uint32_t addr, uint32_t rank)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(mapa_shared(addr, rank))
                 : "memory");
    return v;
}

// Eight consecutive columns (row, col) of the cluster's S partial tiles.
__device__ __forceinline__ void sum_partials(uint32_t part, int row, int col, uint32_t S, float (&z)[8])
{
    const uint32_t at = part + (row * 128 + col) * 4;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        z[i] = 0.f;
#pragma unroll 4
    for (uint32_t s = 0; s < S; ++s) {
        const float4 a = ld_partial(at, s), b = ld_partial(at + 16, s);
        z[0] += a.x, z[1] += a.y, z[2] += a.z, z[3] += a.w;
        z[4] += b.x, z[5] += b.y, z[6] += b.z, z[7] += b.w;
    }
}

// Eight bf16 of a row, n (1..8) of them inside it.
__device__ __forceinline__ void load_piece(const __nv_bfloat16 *p, int n, float (&f)[8])
{
    if (n == 8 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf_lo(w[i]);
            f[2 * i + 1] = bf_hi(w[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = i < n ? __bfloat162float(p[i]) : 0.f;
    }
}

__device__ __forceinline__ void save_piece(__nv_bfloat16 *M, int64_t off, const float (&f)[8], int n, int64_t limit,
                                           const ErrCtx &err)
{
    store_piece(M, off,
                make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])),
                n, limit, err);
}

// What the epilogue of eight columns of a row reads: scales, bias, and the
// residual or the two halves of preact.
struct PieceReads {
    float scale_a, scale_b[8], scale_u[8], bias[8], a[8], b[8];
};

template <int EPI>
__device__ __forceinline__ void read_piece(const SplitArgs &p, PieceReads &rd, int64_t row, int col, int n, int e)
{
    if (p.epi.scale_a) {
        const int64_t src = p.rows ? p.rows[row] : row;
        rd.scale_a = src >= 0 && src < p.T ? p.epi.scale_a[src] : 0.f;
    }
    if (p.epi.scale_b) {
        const float *s = p.epi.scale_b + e * static_cast<int64_t>(EPI == kSwSwiglu ? 2 * p.N : p.N) + col;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            rd.scale_b[j] = j < n ? s[j] : 0.f;
            if constexpr (EPI == kSwSwiglu)
                rd.scale_u[j] = j < n ? s[p.N + j] : 0.f;
        }
    }
    if constexpr (EPI == kSwDense) {
        if (p.epi.bias) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                rd.bias[j] = j < n ? p.epi.bias[col + j] : 0.f;
        }
        if (p.epi.residual)
            load_piece(static_cast<const __nv_bfloat16 *>(p.epi.residual) + row * p.epi.ld_residual + col, n, rd.a);
    }
    if constexpr (EPI == kSwSwigluGrad) {
        const __nv_bfloat16 *P = static_cast<const __nv_bfloat16 *>(p.epi.preact) + row * p.epi.ld_preact + col;
        load_piece(P, n, rd.a);
        load_piece(P + p.N, n, rd.b);
    }
}

template <int IN, int EPI>
__global__ void __launch_bounds__(kSplitThreads, 1) split_kernel(const __grid_constant__ SplitArgs p, ErrCtx err)
{
    constexpr int KB = kb_elems(IN);
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + p.ring_bytes);
    uint64_t *empty = full + kSplitMaxStages;
    uint64_t *done = empty + kSplitMaxStages;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *row_numbers = reinterpret_cast<int *>(smem + p.ring_bytes + kSplitBars - 1024);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = cluster_ctarank(), S = cluster_size();
    const int tile = blockIdx.x / S;
    constexpr int OUT = EPI == kSwSwiglu ? 64 : 128;           // output columns of a tile
    const int tiles_n = ceil_div(p.N, OUT), num_kb = ceil_div(p.K, KB);

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
        tma_prefetch_desc(lane ? &p.tmX : &p.tmW);
    if (warp == 1) {
        tmem_alloc(tmem_slot, p.tmem_cols);
        tmem_relinquish();
    }
    grid_release();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // This cluster's tile (the grid is an upper bound): group, rows, columns.
    // Every warp finds it from the offsets by itself.
    int e = 0, row0 = 0, rows = 0, tn = 0;
    bool work = false;
    auto take = [&](int group, int first, int end, int t) {
        work = true;
        e = group;
        tn = t % tiles_n;
        row0 = first + t / tiles_n * p.w;
        rows = min(p.w, end - row0);
    };
    if constexpr (EPI == kSwDense) {
        if (tile < ceil_div(p.R, p.w) * tiles_n)
            take(0, 0, p.R, tile);
    } else {
        grid_wait();
        int before = 0;              // tiles of the groups before
        for (int e0 = 0; e0 < p.E && !work; e0 += 32) {
            int a = 0, b = 0;
            if (e0 + lane < p.E) {
                a = min(max(p.offsets[e0 + lane], 0), p.R);
                b = min(max(p.offsets[e0 + lane + 1], 0), p.R);
            }
            int inc = ceil_div(max(b - a, 0), p.w) * tiles_n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o)
                    inc += x;
            }
            const uint32_t past = __ballot_sync(0xffffffffu, tile < before + inc);
            const int l = past ? __ffs(past) - 1 : 31;
            const int start = l ? __shfl_sync(0xffffffffu, inc, l - 1) : 0;
            a = __shfl_sync(0xffffffffu, a, l);
            b = __shfl_sync(0xffffffffu, b, l);
            if (past)
                take(e0 + l, a, b, tile - before - start);
            before += __shfl_sync(0xffffffffu, inc, 31);
        }
    }
    const int wt = (rows + 15) & ~15;                          // MMA width
    const int kb0 = static_cast<int>(static_cast<int64_t>(num_kb) * rank / S);
    const int kb1 = static_cast<int>(static_cast<int64_t>(num_kb) * (rank + 1) / S);
    const uint32_t part = smem_u32(smem);                      // the partial tile, over the ring
    if constexpr (EPI == kSwDense)                             // all up to here depends on sizes only
        grid_wait();

    int stage = 0, issued = 0;
    uint32_t phase = 0;
    if (work && (warp == 0 || warp == 2)) {
        // ------------------ TMA producers: the weights (warp 0), the rows (warp 2)
        if (warp == 2 && p.gather) {
            for (int i = lane; i < wt; i += 32) {
                int r = p.map_rows;                            // past the last row: zeros
                if (i < rows) {
                    r = p.rows[row0 + i];
                    r = r < 0 || r >= p.map_rows ? p.map_rows : r;
                }
                row_numbers[i] = r;
            }
            __syncwarp();
        }
        const uint32_t tx = 16384u + static_cast<uint32_t>(p.gather ? wt : p.w) * 128u;
        const int n0 = tn * OUT;
        for (int kb = kb0; kb < kb1; ++kb, ++issued) {
            if (!mbar_wait_warp(&empty[stage], phase ^ 1u, err, abort_flag, kSiteProducerEmpty))
                break;
            uint8_t *sw = smem + stage * p.stage_bytes, *sx = sw + 16384;
            if (warp == 0) {
                mbar_arrive_expect_tx_w(&full[stage], tx);
                if constexpr (EPI == kSwSwiglu) {
                    tma_load_3d_w(sw, &p.tmW, &full[stage], kb * KB, n0, e);
                    tma_load_3d_w(sw + 8192, &p.tmW, &full[stage], kb * KB, p.half_rows + n0, e);
                } else if (p.maj) {
                    tma_load_3d_w(sw, &p.tmW, &full[stage], n0, kb * KB, e);
                    tma_load_3d_w(sw + kMnBoxBytes, &p.tmW, &full[stage], n0 + kMnBox, kb * KB, e);
                } else {
                    tma_load_3d_w(sw, &p.tmW, &full[stage], kb * KB, n0, e);
                }
            } else if (p.gather) {
                for (int i = lane; i < wt / 4; i += 32)
                    tma_gather4(smem_u32(sx) + i * 512, &p.tmX, &full[stage], kb * KB,
                                reinterpret_cast<const int4 *>(row_numbers)[i]);
                __syncwarp();
            } else {
                tma_load_2d_w(sx, &p.tmX, &full[stage], kb * KB, row0);
            }
            if (++stage == p.stages) {
                stage = 0;
                phase ^= 1u;
            }
        }
    } else if (work && warp == 1) {
        // -------------------------------------------- MMA issuer
        const uint32_t idesc = (IN == kInE4m3 ? idesc_e4m3_f32(128, wt) : idesc_bf16_f32(128, wt)) | (p.maj ? 1u << 15 : 0u);
        const uint64_t astep = (p.maj ? kMnKStepBytes : 32) >> 4;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!mbar_wait_warp(&full[stage], phase, err, abort_flag, kSiteMmaFull))
                break;
            tc_fence_after();
            const uint32_t w_s = smem_u32(smem + stage * p.stage_bytes);
            const uint64_t adesc = p.maj ? sdesc_mnmajor_sw128(w_s) : sdesc_kmajor_sw128(w_s);
            const uint64_t bdesc = sdesc_kmajor_sw128(w_s + 16384);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if constexpr (IN == kInE4m3)
                    mma_e4m3_w(tmem, adesc + k * astep, bdesc + k * 2, idesc, (kb != kb0) || (k != 0));
                else
                    mma_bf16_w(tmem, adesc + k * astep, bdesc + k * 2, idesc, (kb != kb0) || (k != 0));
            }
            mma_commit_w(&empty[stage]);
            if (++stage == p.stages) {
                stage = 0;
                phase ^= 1u;
            }
        }
        mma_commit_w(done);
    }
    // The rows of this CTA's share, in eight-column pieces, the warps that are
    // free first.  Their epilogue operands are read ahead of the sum.
    constexpr int PER = OUT / 8;
    const int r_begin = static_cast<int>(static_cast<int64_t>(rows) * rank / S);
    const int r_end = static_cast<int>(static_cast<int64_t>(rows) * (rank + 1) / S);
    const int item0 = (threadIdx.x + kSplitThreads - 64) % kSplitThreads, items = work ? (r_end - r_begin) * PER : 0;
    PieceReads rd;
    auto read = [&](int i) {
        const int col = tn * OUT + i % PER * 8;
        if (i < items && col < p.N)
            read_piece<EPI>(p, rd, row0 + r_begin + i / PER, col, min(8, p.N - col), e);
    };
    if (warp >= 2)
        read(item0);
    if (work && warp >= 2) {
        // ------------------------- the accumulator to the partial tile [row of A][128]
        if (mbar_wait_warp(done, 0, err, abort_flag, kSiteEpiTmemFull)) {
            tc_fence_after();
            const int q = warp & 3;
            for (int c = (warp - 2) / 4; c * 32 < wt; c += 2) {
                uint32_t r[32];
                tmem_ld32(tmem + (static_cast<uint32_t>(q * 32) << 16) + c * 32, r);
                const uint32_t at = part + (c * 32 * 128 + q * 32 + lane) * 4;
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (c * 32 + j < rows)
                        asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + j * 512), "r"(kb0 < kb1 ? r[j] : 0u) : "memory");
            }
            tc_fence_before();
        }
    }
    __syncwarp();
    cluster_sync();                  // every CTA's partial tile is written
    if (work && warp < 2 && *abort_flag) {
        if (warp == 0)               // rows and weights share the stages' barriers
            settle(full, p.stages, stage, phase, issued, err.word, err.budget_ns);
        else
            settle(done, 1, 0, 1, 1, err.word, err.budget_ns);
        __syncwarp();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, p.tmem_cols);
    }
    if (work) {
        // ------------------------- this CTA's share of the rows: sum, epilogue
        __nv_bfloat16 *D = static_cast<__nv_bfloat16 *>(p.D);
        __nv_bfloat16 *P = static_cast<__nv_bfloat16 *>(p.epi.preact);
        const int64_t dcols = EPI == kSwSwigluGrad ? 2ll * p.N : p.N;
        const int64_t d_limit = (p.R - 1) * p.ldd + dcols;
        const int64_t p_limit = (p.R - 1) * p.epi.ld_preact + (EPI == kSwDense ? p.N : 2ll * p.N);
        for (int i = item0; i < items; i += kSplitThreads) {
            const int r = r_begin + i / PER, c = i % PER * 8, col = tn * OUT + c, n = min(8, p.N - col);
            if (n <= 0)
                continue;
            if (warp < 2 || i != item0)
                read(i);
            const int64_t row = row0 + r;
            float z[8], u[8];
            sum_partials(part, r, c, S, z);
            if constexpr (EPI == kSwSwiglu)
                sum_partials(part, r, 64 + c, S, u);
            if (p.epi.scale_a) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    z[j] *= rd.scale_a;
                    if constexpr (EPI == kSwSwiglu)
                        u[j] *= rd.scale_a;
                }
            }
            if (p.epi.scale_b) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    z[j] *= rd.scale_b[j];
                    if constexpr (EPI == kSwSwiglu)
                        u[j] *= rd.scale_u[j];
                }
            }
            if constexpr (EPI == kSwDense) {
                if (p.epi.bias) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        z[j] += rd.bias[j];
                }
                if (P)
                    save_piece(P, row * p.epi.ld_preact + col, z, n, p_limit, err);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    z[j] = p.epi.act == kActRelu   ? act_f<kActRelu>(z[j])
                           : p.epi.act == kActSilu ? act_f<kActSilu>(z[j])
                           : p.epi.act == kActGelu ? act_f<kActGelu>(z[j])
                                                   : z[j];
                if (p.epi.residual) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        z[j] += rd.a[j];
                }
            } else if constexpr (EPI == kSwSwiglu) {
                if (P) {
                    save_piece(P, row * p.epi.ld_preact + col, z, n, p_limit, err);
                    save_piece(P, row * p.epi.ld_preact + p.N + col, u, n, p_limit, err);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    z[j] = silu_f(z[j]) * u[j];
            } else if constexpr (EPI == kSwSwigluGrad) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    swiglu_grad(z[j], rd.a[j], rd.b[j], z[j], u[j]);
                save_piece(D, row * p.ldd + p.N + col, u, n, d_limit, err);
            }
            save_piece(D, row * p.ldd + col, z, n, d_limit, err);
        }
    }
    __syncwarp();
    cluster_sync();                  // no CTA leaves while its partials may be read
}

template <int IN, int EPI>
cudaError_t launch_split_as(const SplitArgs &a, int cluster, int tiles, const ErrCtx &err, cudaStream_t s)
{
    auto kern = split_kernel<IN, EPI>;
    const int smem = 1024 + a.ring_bytes + kSplitBars;
    const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(kern), smem);
    if (e != cudaSuccess)
        return e;
    return launch_overlapped(kern, dim3(static_cast<unsigned>(tiles * cluster)), kSplitThreads, smem, cluster, s, a, err);
}

}  // namespace
}  // namespace tmg
