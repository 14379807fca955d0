// swap_kernel.cuh — the product kernel of the expert-grouped and the dense
// calls: Dᵀ = B · Aᵀ on CTA pairs, operands swapped.  The MMA's M dimension
// (256 rows over a pair) runs over the weight rows, which tile evenly; the
// rows of A (tokens) become the MMA's N, whose width is an operand of the
// instruction: each tile takes the next multiple of 32 of the rows its group
// has, 32 to 256.  A group of 300 rows costs two tiles of 160 columns instead
// of two of 256 rows, a group of 3 one of 32, and no tile crosses a group.
//
// Work.  The group offsets are read on the device: every CTA scans them into
// a table of tile numbers, so the host never waits for the routing.  Within a
// group the tiles go in bands of `group` row tiles, row tiles fastest, so that
// the pairs running together share weight tiles and A panels in L2.  Each pair
// takes the next whole tile as it gets free (feed.cuh); where few tiles would be
// left for the last wave, those are cut along K over several pairs first
// (swap_time) and summed from fp32 partials in pair order: results do not depend
// on timing.
//
// Operands.  Weights: K-major through a 3-D map (K, N, E), or MN-major (N, K,
// E) in 64 x 64 boxes; out-of-range rows and K read as zeros, per expert, so a
// neighbour's values never enter.  For SwiGLU a 5-D map (K, 8, 2, F/8, E)
// lays eight gate rows and their eight up rows next to each other in the tile,
// so gate and up of one column end in the same thread.  A: boxes of 16 to 128
// rows, or, with `gather`, TMA gathers of four named rows each (an index out of
// range reads zeros).  A gather takes 46 ns of an SM's TMA unit, so this is for
// tiles of at most 64 rows (8 gathers a K block and CTA, the 0.37 us that the
// block's weights take from HBM); for wider tiles the caller copies the rows
// first (65528 x 2048 x 2048: 1263 us gathered here, 390 copied, of them 45 for
// the copy).  Rows of the next group that a box brings along give columns that
// no one reads.
//
// Roles per CTA (eleven warps): 0 TMA producer, 1 MMA issuer (CTA 0 of the
// pair) and TMEM owner, 2..9 epilogue, two warps per TMEM lane quarter taking
// 32-column chunks in turn, 10 the tile feed.  The accumulator is double-buffered
// (2 x 256 columns).  Lanes are output columns and registers are rows there, so
// the epilogue reads 16x256b fragments, whose pairs stmatrix transposes into a
// 2 KB tile per warp; D, preact and the residual move in 16-byte pieces.
//
// What bounds it.  Wide tiles: the operands' way into the SMs, 13 - 14.5 TB/s,
// with the tensor pipe busy 73 - 81 % (8191 x 4096 x 4096 143 us, with bias, GELU,
// residual and preact 164; 65528 rows over 64 groups, 2048 x 2048, 341 us, 1.61
// PFLOP/s).  Few rows a group: the weights' bytes (488 rows over 64 groups, 271 MB,
// 45.4 us, 5.9 TB/s).
#pragma once

#include "act.cuh"
#include "feed.cuh"
#include "grouped.h"
#include "launch.cuh"
#include "pieces.cuh"
#include "staging.cuh"
#include "tc2_kernel.cuh"

namespace tmg {

// Epilogue families (template parameter EPI).
enum { kSwPlain = 0, kSwDense = 1, kSwSwiglu = 2, kSwSwigluGrad = 3 };

struct SwapArgs {
    CUtensorMap tmW;
    CUtensorMap tmX[4];        // boxes of 16, 32, 64, 128 rows; gather: tmX[0], one row
    CUtensorMap tmD, tmP;      // dense: D and preact, boxes of 32 columns x 32 rows
    int tma_d, tma_p;          // they are there
    int staging;               // bytes of a warp's staging tiles
    void *D;
    const int32_t *offsets, *rows;
    ProductEpi epi;
    int64_t ldd;
    int R, T, N, K, E;         // N: output columns of the tile grid (F with SwiGLU)
    int maj;                   // weights MN-major
    int gather;                // row r of D is row rows[r] of the map (else its own row)
    int map_rows;              // rows of the map
    int maxw;                  // widest tile, a multiple of 32
    int stages, stage_bytes;
    int group;                 // row tiles per band
    float block_ns;            // a K block of a tile of maxw columns
    float hbm_ns;              // HBM's time for the weights, a tile's share
    float *partials;           // sw_partial_floats(maxw) per pair; null: no tile is split
    uint32_t *counters;        // 16 per cut tile
    uint32_t *feed;            // the tile counter
};

constexpr int kSwMaxW = 256;
// fp32 partials of a pair's piece: 2 CTAs, 4 lane quarters of 32 x maxw
__host__ __device__ inline int64_t sw_partial_floats(int maxw) { return 2ll * 4 * 32 * maxw; }
constexpr int kSwStage = 2048;       // a warp's staging tile: two of them for the dense product's TMA stores
constexpr int kSwMaxStages = 12;
constexpr int kSwGatherW = 64;       // widest tile with gathers
constexpr int kSwBars = (2 * kSwMaxStages + 4) * 8 + sizeof(FeedSmem) + 16 + kSwGatherW * 2;  // barriers, feed, TMEM address, abort flag, row numbers
__host__ __device__ inline int sw_box_rows(int half) { return half <= 16 ? 16 : half <= 32 ? 32 : half <= 64 ? 64 : 128; }
__host__ inline int sw_smem(int stages, int stage_bytes, int staging, int E)
{
    return 1024 + stages * stage_bytes + 8 * staging + kSwBars + 8 * (E + 1);
}

// Nanoseconds that `total` tiles of w columns take over np pairs, and how the last
// wave is split (tail): where at most half the pairs have a tile in it, each of
// its tiles is cut along K over 2 to 8 pairs, before their whole tiles, so that
// the sums are under way while those run.  A cut adds swap_cut_ns (measured at 128
// to 256 columns).  2489 x 5648 x 8192, 230 tiles: 151 us whole, 127 with two tiles
// over eight pairs each; 875 x 6064 x 5920, 96 tiles: 52.8 and 42.6.  block_ns: a K
// block of a tile; hbm_ns: the time of the weights' bytes.
struct SwapTail {
    int tiles, each;           // tiles that are cut, pieces of each
};
__host__ __device__ inline float swap_cut_ns(int w, int each)
{
    return 2500.f + w * (1.f / 256.f) * (4000.f + 600.f * each);
}
// Only where half a tile is worth more than a cut in two: shorter ones would gain
// little by more pieces (2489 x 5648 x 3000 75.4 us whole, 79.6 cut; 5486 x 6192 x
// 2896 117 and 115).
__host__ __device__ inline bool swap_may_cut(int num_kb, int w, float block_ns)
{
    return num_kb * block_ns * 0.5f > swap_cut_ns(w, 2);
}
__host__ __device__ inline float swap_time(int total, int np, int num_kb, int w, float block_ns, float hbm_ns, SwapTail &tail)
{
    const int q = total / np, rem = total - q * np;
    const float tile = num_kb * block_ns;
    const float whole = (q + (rem ? 1 : 0)) * tile;
    const float best = whole > hbm_ns ? whole : hbm_ns;
    const int each = rem == 0 ? 0 : np / rem < 8 ? np / rem : 8;
    tail.tiles = 0;
    tail.each = 1;
    if (each < 2 || num_kb < each || !swap_may_cut(num_kb, w, block_ns))
        return best;
    const float shared = q * tile + tile / each;
    const float cut = (shared > hbm_ns ? shared : hbm_ns) + swap_cut_ns(w, each);
    if (cut >= best)
        return best;
    tail.tiles = rem;
    tail.each = each;
    return cut;
}

cudaError_t launch_swap(const SwapArgs &a, int epi, bool e4m3, int num_sms, const ErrCtx &err, cudaStream_t s);

namespace {

// 3-D and 5-D tile loads and the four-row gather, into this CTA's shared
// memory, counted on an mbarrier of the pair's CTA 0.
__device__ __forceinline__ void tma_load_3d_pair_w(void *dst, const CUtensorMap *map, uint32_t bar, int c0, int c1, int c2)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];\n\t}" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

__device__ __forceinline__ void tma_load_5d_pair_w(void *dst, const CUtensorMap *map, uint32_t bar, int c0, int c3, int c4)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %4, %5, %6}], [%2];\n\t}" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(0), "r"(c3), "r"(c4)
        : "memory");
}

__device__ __forceinline__ void tma_gather4_pair(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, const int4 &r)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes.cta_group::2"
                 " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w)
                 : "memory");
}

// 32 lanes x 32 columns of the accumulator as matrix fragments: v[16 h + 4 g +
// 2 s + b] is lane 16 h + 8 s + t/4, column 8 g + 2 (t mod 4) + b.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, float (&v)[32])
{
    uint32_t r[32];
#pragma unroll
    for (int h = 0; h < 2; ++h)
        asm volatile(
            "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
            "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
            : "=r"(r[16 * h + 0]), "=r"(r[16 * h + 1]), "=r"(r[16 * h + 2]), "=r"(r[16 * h + 3]), "=r"(r[16 * h + 4]),
              "=r"(r[16 * h + 5]), "=r"(r[16 * h + 6]), "=r"(r[16 * h + 7]), "=r"(r[16 * h + 8]), "=r"(r[16 * h + 9]),
              "=r"(r[16 * h + 10]), "=r"(r[16 * h + 11]), "=r"(r[16 * h + 12]), "=r"(r[16 * h + 13]),
              "=r"(r[16 * h + 14]), "=r"(r[16 * h + 15])
            : "r"(taddr + (static_cast<uint32_t>(16 * h) << 16))
            : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i)
        v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void stmatrix4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}

__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t &a, uint32_t &b, uint32_t &c, uint32_t &d)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
                 : "r"(addr)
                 : "memory");
}

// The warp's staging tile: 32 rows of COLS bf16 (COLS = 32 or 16), 16-byte
// pieces swizzled so that the eight rows of a matrix touch different banks.
template <int COLS>
__device__ __forceinline__ uint32_t stage_addr(uint32_t base, int row, int piece)
{
    if constexpr (COLS == 32)
        return base + row * 64 + ((piece ^ ((row >> 1) & 3)) << 4);
    else
        return base + row * 32 + ((piece ^ ((row >> 2) & 1)) << 4);
}

// Fragment words -> the staging tile.  COLS = 32: w[4 g + m], matrix m the
// columns 8 m .. 8 m + 7, g the rows 8 g ..; COLS = 16: w[2 g + m].
template <int COLS>
__device__ __forceinline__ void stage_frag(uint32_t base, int lane, const uint32_t *w)
{
    if constexpr (COLS == 32) {
#pragma unroll
        for (int g = 0; g < 4; ++g)
            stmatrix4_trans(stage_addr<32>(base, 8 * g + (lane & 7), lane >> 3), w[4 * g], w[4 * g + 1], w[4 * g + 2],
                            w[4 * g + 3]);
    } else {
#pragma unroll
        for (int g = 0; g < 4; g += 2)
            stmatrix4_trans(stage_addr<16>(base, 8 * (g + (lane >> 4)) + (lane & 7), (lane >> 3) & 1), w[2 * g], w[2 * g + 1],
                            w[2 * g + 2], w[2 * g + 3]);
    }
}

// The staging tile -> rows r0 .. r0 + nt - 1, columns n0 .. of a row-major
// matrix with `cols` columns.
template <int COLS>
__device__ __forceinline__ void store_staged(uint32_t base, int lane, __nv_bfloat16 *M, int64_t ld, int64_t r0, int nt, int n0,
                                             int cols, int64_t limit, const ErrCtx &err)
{
    constexpr int PER = COLS / 8;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int u = i * 32 + lane, row = u / PER, piece = u % PER;
        const int n = n0 + piece * 8;
        const uint4 v = lds128(stage_addr<COLS>(base, row, piece));
        if (row >= nt || n >= cols)
            continue;
        store_piece(M, (r0 + row) * ld + n, v, min(8, cols - n), limit, err);
    }
}

// A warp's staging tiles.  With results stored by TMA (the dense product's, whose
// maps end with its rows) there are two, used in turn: one is filled while the
// store of the other still reads it.
struct Staging {
    uint32_t base, turn;
    bool tma;

    __device__ __forceinline__ uint32_t tile() const { return base + (tma ? (turn & 1) * kSwStage : 0); }
    // The current tile may be written.
    __device__ __forceinline__ void acquire() const
    {
        if (tma) {
            if ((threadIdx.x & 31) == 0)
                asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
            __syncwarp();
        }
    }
};

// A chunk's fragment words to rows r0 .., columns n0 .. of a matrix.
template <int COLS>
__device__ __forceinline__ void put_frag(const Staging &st, int lane, const uint32_t *w, __nv_bfloat16 *M, int64_t ld, int64_t r0,
                                         int nt, int n0, int cols, int64_t limit, const ErrCtx &err)
{
    stage_frag<COLS>(st.base, lane, w);
    __syncwarp();
    store_staged<COLS>(st.base, lane, M, ld, r0, nt, n0, cols, limit, err);
    __syncwarp();
}

// The same by TMA where the matrix has a map.
__device__ __forceinline__ void put_dense(Staging &st, int lane, const uint32_t *w, const CUtensorMap *map, __nv_bfloat16 *M,
                                          int64_t ld, int64_t r0, int nt, int n0, int cols, int64_t limit, const ErrCtx &err)
{
    st.acquire();
    stage_frag<32>(st.tile(), lane, w);
    if (map) {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
            if (n0 < cols && nt > 0)
                asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                                 reinterpret_cast<uint64_t>(map)),
                             "r"(n0), "r"(static_cast<int>(r0)), "r"(st.tile())
                             : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
        ++st.turn;
    } else {
        __syncwarp();
        store_staged<32>(st.tile(), lane, M, ld, r0, nt, n0, cols, limit, err);
        __syncwarp();
    }
}

// 32 rows x 32 columns of a row-major matrix, zeros outside, in two steps:
// the loads (four 16-byte pieces per lane, issued early), and the way through
// the staging tile to fragment words.
__device__ __forceinline__ void load_rows(uint4 (&v)[4], int lane, const __nv_bfloat16 *M, int64_t ld, int64_t r0, int nt,
                                          int n0, int cols)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int u = i * 32 + lane, row = u / 4;
        const int n = n0 + u % 4 * 8;
        v[i] = make_uint4(0, 0, 0, 0);
        if (row < nt && n < cols) {
            const __nv_bfloat16 *p = M + (r0 + row) * ld + n;
            if (cols - n >= 8 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
                v[i] = *reinterpret_cast<const uint4 *>(p);
            } else {
                uint32_t u4[4] = {};
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (n + j < cols)
                        u4[j / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(p)[j]) << (16 * (j & 1));
                v[i] = make_uint4(u4[0], u4[1], u4[2], u4[3]);
            }
        }
    }
}

__device__ __forceinline__ void rows_frag(uint32_t base, int lane, const uint4 (&v)[4], uint32_t (&w)[16])
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        sts128(stage_addr<32>(base, (i * 32 + lane) / 4, lane % 4), v[i]);
    __syncwarp();
#pragma unroll
    for (int g = 0; g < 4; ++g)
        ldmatrix4_trans(stage_addr<32>(base, 8 * g + (lane & 7), lane >> 3), w[4 * g], w[4 * g + 1], w[4 * g + 2], w[4 * g + 3]);
    __syncwarp();
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Fragment values -> words: matrix m = 2 h + s of group g.
__device__ __forceinline__ void pack_frag(const float (&v)[32], uint32_t (&w)[16])
{
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const int i = 16 * (m >> 1) + 4 * g + 2 * (m & 1);
            w[4 * g + m] = pack_bf16x2(v[i], v[i + 1]);
        }
}

// One 32-row x 32-lane chunk of a finished sum: the epilogue and the stores.
// n0: the first output column of the warp's lanes (SwiGLU: 16 columns);
// sb: scale_b of this thread's four lanes (index 2 h + s), bias likewise;
// sa_lane: scale_a of row `lane` of the chunk; pre: the chunk's residual, or the
// two halves of preact that swiglu_grad reads.
struct EpiReads {
    uint4 a[4], b[4];
};

// Issue a chunk's epilogue reads (ahead of the sum that they meet).
template <int EPI>
__device__ __forceinline__ void read_ahead(const SwapArgs &p, EpiReads &pre, int lane, int64_t r0, int nt, int n0)
{
    if constexpr (EPI == kSwDense) {
        if (p.epi.residual)
            load_rows(pre.a, lane, static_cast<const __nv_bfloat16 *>(p.epi.residual), p.epi.ld_residual, r0, nt, n0, p.N);
    }
    if constexpr (EPI == kSwSwigluGrad) {
        const __nv_bfloat16 *P = static_cast<const __nv_bfloat16 *>(p.epi.preact);
        load_rows(pre.a, lane, P, p.epi.ld_preact, r0, nt, n0, p.N);
        load_rows(pre.b, lane, P + p.N, p.epi.ld_preact, r0, nt, n0, p.N);
    }
}

template <int EPI, class Ahead>
__device__ __forceinline__ void finish_chunk(const SwapArgs &p, float (&v)[32], Staging &stg, int lane, int64_t r0, int nt,
                                             int n0, float sa_lane, const float (&sb)[4], const float (&bias)[4],
                                             EpiReads &pre, Ahead &&ahead, const ErrCtx &err)
{
    __nv_bfloat16 *D = static_cast<__nv_bfloat16 *>(p.D);
    __nv_bfloat16 *P = static_cast<__nv_bfloat16 *>(p.epi.preact);
    const int64_t dcols = EPI == kSwSwigluGrad ? 2ll * p.N : p.N;
    const int64_t d_limit = (p.R - 1) * p.ldd + dcols;
    const int64_t p_limit = (p.R - 1) * p.epi.ld_preact + (EPI == kSwDense ? p.N : 2ll * p.N);
    if (p.epi.scale_a) {
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const float f = __shfl_sync(0xffffffffu, sa_lane, 8 * g + 2 * (lane & 3) + b);
#pragma unroll
                for (int m = 0; m < 4; ++m)
                    v[16 * (m >> 1) + 4 * g + 2 * (m & 1) + b] *= f;
            }
    }
    if (p.epi.scale_b) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            v[i] *= sb[2 * (i >> 4) + ((i >> 1) & 1)];
    }
    uint32_t w[16];
    if constexpr (EPI == kSwPlain) {
        pack_frag(v, w);
        put_frag<32>(stg, lane, w, D, p.ldd, r0, nt, n0, p.N, d_limit, err);
    } else if constexpr (EPI == kSwDense) {
        if (p.epi.bias) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                v[i] += bias[2 * (i >> 4) + ((i >> 1) & 1)];
        }
        if (P) {
            pack_frag(v, w);
            put_dense(stg, lane, w, p.tma_p ? &p.tmP : nullptr, P, p.epi.ld_preact, r0, nt, n0, p.N, p_limit, err);
        }
        if (p.epi.act == kActRelu) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                v[i] = act_f<kActRelu>(v[i]);
        } else if (p.epi.act == kActSilu) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                v[i] = act_f<kActSilu>(v[i]);
        } else if (p.epi.act == kActGelu) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                v[i] = act_f<kActGelu>(v[i]);
        }
        if (p.epi.residual) {
            stg.acquire();
            rows_frag(stg.tile(), lane, pre.a, w);
            ahead();
#pragma unroll
            for (int g = 0; g < 4; ++g)
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int i = 16 * (m >> 1) + 4 * g + 2 * (m & 1);
                    v[i] += bf_lo(w[4 * g + m]);
                    v[i + 1] += bf_hi(w[4 * g + m]);
                }
        }
        pack_frag(v, w);
        put_dense(stg, lane, w, p.tma_d ? &p.tmD : nullptr, D, p.ldd, r0, nt, n0, p.N, d_limit, err);
    } else if constexpr (EPI == kSwSwiglu) {
        // lanes 16 h + t/4 are gates, 16 h + 8 + t/4 their ups; column n0 + 8 h + t/4
        uint32_t x[8];
        if (P) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
#pragma unroll
                for (int g = 0; g < 4; ++g)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        x[2 * g + h] = pack_bf16x2(v[16 * h + 4 * g + 2 * s], v[16 * h + 4 * g + 2 * s + 1]);
                // columns past F of the gate half belong to the up half: the
                // bound is the half's own, the second half starts at F
                put_frag<16>(stg, lane, x, P + s * static_cast<int64_t>(p.N), p.epi.ld_preact, r0, nt, n0, p.N,
                             p_limit - s * static_cast<int64_t>(p.N), err);
            }
        }
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = 16 * h + 4 * g;
                x[2 * g + h] = pack_bf16x2(silu_f(v[i]) * v[i + 2], silu_f(v[i + 1]) * v[i + 3]);
            }
        put_frag<16>(stg, lane, x, D, p.ldd, r0, nt, n0, p.N, d_limit, err);
    } else {
        uint32_t u[16];
        rows_frag(stg.base, lane, pre.a, w);
        rows_frag(stg.base, lane, pre.b, u);
        ahead();
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const int i = 16 * (m >> 1) + 4 * g + 2 * (m & 1), k = 4 * g + m;
                float g0, g1, u0, u1;
                swiglu_grad(v[i], bf_lo(w[k]), bf_lo(u[k]), g0, u0);
                swiglu_grad(v[i + 1], bf_hi(w[k]), bf_hi(u[k]), g1, u1);
                w[k] = pack_bf16x2(g0, g1);
                u[k] = pack_bf16x2(u0, u1);
            }
        put_frag<32>(stg, lane, w, D, p.ldd, r0, nt, n0, p.N, d_limit, err);
        put_frag<32>(stg, lane, u, D + p.N, p.ldd, r0, nt, n0, p.N, d_limit - p.N, err);
    }
}

// A tile: its group, first row, rows, MMA width and weight tile.
struct SwapTile {
    int e, row0, rows, w, tn;
};

__device__ __forceinline__ SwapTile swap_tile(int t, const int *off, const int *start, int E, int maxw, int tiles_n, int group)
{
    int lo = 0, hi = E;              // the last group that starts at or before t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= t)
            lo = mid;
        else
            hi = mid;
    }
    SwapTile x;
    x.e = lo;
    const int first = off[lo], rows = off[lo + 1] - first, tiles = ceil_div(rows, maxw);
    int tm;
    tile_coords(t - start[lo], tiles, tiles_n, group, tm, x.tn);
    // the group's rows in 32s, spread evenly over its tiles: the first few
    // take one more
    const int grains = ceil_div(rows, 32), each = grains / tiles, more = grains - each * tiles;
    const int g0 = tm * each + min(tm, more);
    x.w = 32 * (each + (tm < more ? 1 : 0));
    x.row0 = first + 32 * g0;
    x.rows = min(x.w, rows - 32 * g0);
    return x;
}

constexpr int kSwThreads = 352;

// The walk of a pair: its piece of a cut tile, if it has one, then whole tiles.
struct SwapWalk {
    Feed feed;
    int cut, each, num_kb;           // cut tiles, pieces of each
    int c;                           // the pair, or -1 once its piece is taken
    const ErrCtx &err;
    volatile int *abort;

    __device__ SwapWalk(FeedSmem *f, int c_, int nc, int total, const SwapTail &t, int nkb, const ErrCtx &e, volatile int *ab)
        : feed(f, c_, nc, total - t.tiles), cut(t.tiles), each(t.each), num_kb(nkb),
          c(c_ < t.tiles * t.each ? c_ : -1), err(e), abort(ab)
    {
    }

    // Tile, K blocks, and whether they are a piece of a cut tile.
    __device__ __forceinline__ bool next(int &tile, int &kb0, int &kb1, bool &partial)
    {
        partial = c >= 0;
        if (!partial) {
            kb0 = 0;
            kb1 = num_kb;
            const bool more = feed.next(tile, err, abort);
            tile += cut;
            return more;
        }
        tile = c / each;
        const int i = c - tile * each;
        kb0 = static_cast<int>(static_cast<int64_t>(num_kb) * i / each);
        kb1 = static_cast<int>(static_cast<int64_t>(num_kb) * (i + 1) / each);
        c = -1;
        return true;
    }
};

template <int IN, int EPI>
__global__ void __launch_bounds__(kSwThreads, 1) swap_kernel(const __grid_constant__ SwapArgs p, ErrCtx err)
{
    constexpr int KB = kb_elems(IN);
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    uint8_t *staging = smem + p.stages * p.stage_bytes;
    uint64_t *full = reinterpret_cast<uint64_t *>(staging + 8 * p.staging);
    uint64_t *empty = full + kSwMaxStages;
    uint64_t *tfull = empty + kSwMaxStages;
    uint64_t *tempty = tfull + 2;
    FeedSmem *feed_smem = reinterpret_cast<FeedSmem *>(tempty + 2);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(feed_smem + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *row_numbers = reinterpret_cast<int *>(tmem_slot + 4);
    int *off = row_numbers + kSwGatherW / 2, *start = off + p.E + 1;

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = cluster_ctarank();
    const int cluster = blockIdx.x >> 1, nclusters = gridDim.x >> 1;
    constexpr int OUT = EPI == kSwSwiglu ? 128 : 256;          // output columns of a tile
    const int tiles_n = ceil_div(p.N, OUT), num_kb = ceil_div(p.K, KB);

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
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
    if (warp == 0 && lane < (p.gather ? 2 : 5))
        tma_prefetch_desc(lane == 0 ? &p.tmW : &p.tmX[lane - 1]);
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, 512);
        tmem_relinquish_pair();
    }
    grid_release();
    if constexpr (EPI != kSwDense)
        grid_wait();
    for (int i = threadIdx.x; i <= p.E; i += kSwThreads)
        off[i] = EPI != kSwDense ? min(max(p.offsets[i], 0), p.R) : (i ? p.R : 0);
    __syncthreads();
    if (warp == 2) {                 // tiles before each group
        int run = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + lane;
            const int n = e < p.E ? ceil_div(max(off[e + 1] - off[e], 0), p.maxw) * tiles_n : 0;
            int inc = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o)
                    inc += x;
            }
            if (e < p.E)
                start[e] = run + inc - n;
            run += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0)
            start[p.E] = run;
    }
    tc_fence_before();
    cluster_sync();          // barriers of both CTAs initialised, TMEM allocated, tables written
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    const int total = start[p.E];
    SwapTail tail{0, 1};
    if (p.partials)
        swap_time(total, nclusters, num_kb, p.maxw, p.block_ns, total * p.hbm_ns, tail);
    SwapWalk walk(feed_smem, cluster, nclusters, total, tail, num_kb, err, abort_flag);
    int tile, kb0, kb1;
    bool partial;
    // The dense product's tiles depend on sizes only: its warps wait for the
    // preceding kernel after their first tile is decoded (4096 x 4096 x 4096 in a
    // row: 80.6 -> 77.1 us).

    if (warp == 0) {
        // ---------------------------------------------- TMA producer
        int stage = 0;
        uint32_t phase = 0;
        int64_t issued = 0;
        bool ok = true;
        walk.feed.producer = rank == 0;
        while (ok && walk.next(tile, kb0, kb1, partial)) {
            const SwapTile x = swap_tile(tile, off, start, p.E, p.maxw, tiles_n, p.group);
            if constexpr (EPI == kSwDense)
                grid_wait();
            const int half = x.w / 2, xrow = x.row0 + static_cast<int>(rank) * half;
            const int box = sw_box_rows(half);
            const CUtensorMap *tmx = &p.tmX[p.gather || box == 16 ? 0 : box == 32 ? 1 : box == 64 ? 2 : 3];
            int4 four = make_int4(0, 0, 0, 0);
            if (p.gather) {
                __syncwarp();
                int r = p.map_rows;             // past the last row: zeros
                if (lane < half && static_cast<int>(rank) * half + lane < x.rows) {
                    r = p.rows[xrow + lane];
                    r = r < 0 || r >= p.map_rows ? p.map_rows : r;
                }
                row_numbers[lane] = r;
                __syncwarp();
                if (lane < half / 4)
                    four = reinterpret_cast<const int4 *>(row_numbers)[lane];
            }
            const uint32_t tx = 2u * (16384u + static_cast<uint32_t>(p.gather ? half : box) * 128u);
            const int n0 = x.tn * OUT + static_cast<int>(rank) * (OUT / 2);
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!mbar_wait_cluster_warp(&empty[stage], phase ^ 1u, err, abort_flag, kSiteProducerEmpty)) {
                    ok = false;
                    break;
                }
                if (rank == 0)
                    mbar_arrive_expect_tx_w(&full[stage], tx);
                const uint32_t bar0 = mapa_shared(smem_u32(&full[stage]), 0);
                uint8_t *sw = smem + stage * p.stage_bytes, *sx = sw + 16384;
                if constexpr (EPI == kSwSwiglu) {
                    tma_load_5d_pair_w(sw, &p.tmW, bar0, kb * KB, n0 / 8, x.e);
                } else if (p.maj) {
                    tma_load_3d_pair_w(sw, &p.tmW, bar0, n0, kb * KB, x.e);
                    tma_load_3d_pair_w(sw + kMnBoxBytes, &p.tmW, bar0, n0 + kMnBox, kb * KB, x.e);
                } else {
                    tma_load_3d_pair_w(sw, &p.tmW, bar0, kb * KB, n0, x.e);
                }
                if (p.gather) {
                    if (lane < half / 4)
                        tma_gather4_pair(smem_u32(sx) + lane * 512, tmx, bar0, kb * KB, four);
                    __syncwarp();
                } else {
                    tma_load_2d_pair_w(sx, tmx, bar0, kb * KB, xrow);
                }
                ++issued;
                if (++stage == p.stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        // Tail: every stage this CTA filled is released (no multicast arrive
        // still on its way here), and in CTA 0 every load of the pair landed.
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
            int local = 0;
            bool ok = true;
            const uint64_t astep = (p.maj ? kMnKStepBytes : 32) >> 4;
            // The next tile is fetched and decoded (0.3 us) while the last K
            // blocks of this one are under way, so the MMAs go on without a gap.
            const uint32_t base = (IN == kInE4m3 ? idesc_e4m3_f32(256, 0) : idesc_bf16_f32(256, 0)) | (p.maj ? 1u << 15 : 0u);
            bool more = walk.next(tile, kb0, kb1, partial);
            int w = more ? swap_tile(tile, off, start, p.E, p.maxw, tiles_n, p.group).w : 0;
            while (ok && more) {
                const uint32_t idesc = base | static_cast<uint32_t>(w >> 3) << 17;
                const int b0 = kb0, b1 = kb1, turn = max(b0, b1 - 3);
                const int acc = local & 1;
                const uint32_t acc_phase = (local >> 1) & 1;
                ++local;
                if (!mbar_wait_cluster_warp(&tempty[acc], acc_phase ^ 1u, err, abort_flag, kSiteMmaTmemEmpty))
                    break;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + acc * kSwMaxW;
                for (int kb = b0; kb < b1; ++kb) {
                    if (kb == turn) {
                        more = walk.next(tile, kb0, kb1, partial);
                        if (more)
                            w = swap_tile(tile, off, start, p.E, p.maxw, tiles_n, p.group).w;
                    }
                    if (!mbar_wait_cluster_warp(&full[stage], phase, err, abort_flag, kSiteMmaFull)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t w_s = smem_u32(smem + stage * p.stage_bytes);
                    const uint64_t adesc = p.maj ? sdesc_mnmajor_sw128(w_s) : sdesc_kmajor_sw128(w_s);
                    const uint64_t bdesc = sdesc_kmajor_sw128(w_s + 16384);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if constexpr (IN == kInE4m3)
                            mma_e4m3_pair_w(d_tmem, adesc + k * astep, bdesc + k * 2, idesc, (kb != b0) || (k != 0));
                        else
                            mma_bf16_pair_w(d_tmem, adesc + k * astep, bdesc + k * 2, idesc, (kb != b0) || (k != 0));
                    }
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
    } else if (warp == 10) {
        if constexpr (EPI == kSwDense)
            grid_wait();
        feed_run(feed_smem, rank, total - tail.tiles, nclusters, p.feed, err, abort_flag);
    } else {
        // ---------------------------------------------------- epilogue
        const int ew = warp - 2, half = ew / 4, q = warp & 3;
        Staging stg{smem_u32(staging + ew * p.staging), 0, p.tma_d || p.tma_p};
        int local = 0;
        while (walk.next(tile, kb0, kb1, partial)) {
            const SwapTile x = swap_tile(tile, off, start, p.E, p.maxw, tiles_n, p.group);
            const int acc = local & 1;
            const uint32_t acc_phase = (local >> 1) & 1;
            ++local;
            const int n0 = x.tn * OUT + static_cast<int>(rank) * (OUT / 2) + q * (OUT / 8);
            if constexpr (EPI == kSwDense)
                grid_wait();
            float sb[4] = {1.f, 1.f, 1.f, 1.f}, bias[4] = {};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // lane 16 h + 8 s + t/4 with i = 2 h + s; SwiGLU: s = 1 is the up half
                const int n = EPI == kSwSwiglu ? n0 + 8 * (i >> 1) + lane / 4 : n0 + 8 * i + lane / 4;
                const int64_t at = EPI == kSwSwiglu ? (i & 1) * static_cast<int64_t>(p.N) + n : n;
                if (n < p.N) {
                    if (p.epi.scale_b)
                        sb[i] = p.epi.scale_b[x.e * static_cast<int64_t>(EPI == kSwSwiglu ? 2 * p.N : p.N) + at];
                    if (EPI == kSwDense && p.epi.bias)
                        bias[i] = p.epi.bias[n];
                }
            }
            const int chunks = x.w / 32;
            EpiReads pre;
            auto ahead = [&](int c) {
                if (c < chunks)
                    read_ahead<EPI>(p, pre, lane, x.row0 + c * 32, min(32, x.rows - c * 32), n0);
            };
            // scale_a of a chunk's row `lane`, read a chunk ahead (but beside the
            // reads of preact, where the registers would spill): 29687 rows of
            // E4M3 by 1456 x 416 46.7 -> 40.0 us
            auto scale_of = [&](int c) {
                const int64_t r = x.row0 + c * 32 + lane;
                if (!p.epi.scale_a || c >= chunks || c * 32 + lane >= x.rows)
                    return 1.f;
                const int src = p.rows ? p.rows[r] : static_cast<int>(r);
                return src >= 0 && src < p.T ? p.epi.scale_a[src] : 0.f;
            };
            float sa_next = EPI == kSwSwigluGrad ? 1.f : scale_of(half);
            if (!partial)
                ahead(half);
            if (!mbar_wait_cluster(&tfull[acc], acc_phase, err, abort_flag, kSiteEpiTmemFull))
                break;
            tc_fence_after();
            const uint32_t tbase = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * kSwMaxW;
            const int64_t piece = 32 * p.maxw;
            const int64_t limit = nclusters * sw_partial_floats(p.maxw);
            bool finish = !partial;
            int c_first = 0, c_last = 0;
            if (partial) {
                const int64_t mine = ((static_cast<int64_t>(cluster) * 2 + rank) * 4 + q) * piece;
#pragma unroll 1
                for (int c = half; c < chunks; c += 2) {
                    float v[32];
                    tmem_ld_frag(tbase + c * 32, v);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int64_t at = mine + ((c * 8 + j) * 32 + lane) * 4;
                        if (span_ok(at, 4, limit, err, kBndPartials))
                            *reinterpret_cast<float4 *>(p.partials + at) =
                                make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_cluster(mapa_shared(smem_u32(&tempty[acc]), 0));
                if (half < chunks) {
                    c_first = tile * walk.each;
                    c_last = c_first + walk.each - 1;
                    const int64_t at = (static_cast<int64_t>(tile) * 2 + rank) * 8 + ew;
                    finish = last_arrival(p.counters + at, c_last - c_first,
                                          bounds_ok(at, 2ll * nclusters * 16, err, kBndCounters));
                }
            }
            if (finish) {
                if (partial)
                    ahead(half);
#pragma unroll 1
                for (int c = half; c < chunks; c += 2) {
                    const int64_t r0 = x.row0 + c * 32;
                    const int nt = min(32, x.rows - c * 32);
                    const float sa = EPI == kSwSwigluGrad ? scale_of(c) : sa_next;
                    if constexpr (EPI != kSwSwigluGrad)
                        sa_next = scale_of(c + 2);
                    float v[32];
                    if (!partial) {
                        tmem_ld_frag(tbase + c * 32, v);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            v[i] = 0.f;
                        add_pieces(v, p.partials, limit, c * 1024 + lane * 4, c_first, c_last, [&](int cc) {
                            return ((static_cast<int64_t>(cc) * 2 + rank) * 4 + q) * piece;
                        }, err);
                    }
                    finish_chunk<EPI>(p, v, stg, lane, r0, nt, n0, sa, sb, bias, pre, [&] { ahead(c + 2); }, err);
                }
            }
            if (!partial) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_cluster(mapa_shared(smem_u32(&tempty[acc]), 0));
            }
        }
        if (stg.tma && lane == 0)
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }

    __syncwarp();
    tc_fence_before();
    cluster_sync();          // no CTA leaves while its peer may still touch it
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 512);
    }
}

template <int IN, int EPI>
cudaError_t launch_swap_as(const SwapArgs &a, int num_sms, const ErrCtx &err, cudaStream_t s)
{
    auto kern = swap_kernel<IN, EPI>;
    const int smem = sw_smem(a.stages, a.stage_bytes, a.staging, a.E);
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(kern), smem);
    if (e != cudaSuccess)
        return e;
    return launch_overlapped(kern, dim3(2 * (num_sms / 2)), kSwThreads, smem, 2, s, a, err);
}

}  // namespace
}  // namespace tmg
