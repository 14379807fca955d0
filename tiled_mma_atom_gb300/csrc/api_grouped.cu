// api_grouped.cu — C ABI of the routing, the expert-grouped products and the
// dense product with the residual epilogue (include/tmg.h): argument checks
// and launches.
#include <algorithm>
#include <cstdio>
#include <cstring>

#include "act.cuh"
#include "grouped.h"
#include "host.h"
#include "product.h"
#include "split.h"
#include "swap_kernel.cuh"
#include "wgrad.h"

namespace tmg {
namespace {

// Common checks of both products; the launch follows in run_product.
tmg_status check_product(const GroupedArgs &a)
{
    if (a.R < 0 || a.N < 0 || a.K < 0 || a.T < 0)
        return fail(TMG_ERR_INVALID_ARG, "negative extent R=%lld N=%lld K=%lld T=%lld", (long long)a.R, (long long)a.N,
                    (long long)a.K, (long long)a.T);
    if (a.R > kMax31 || a.N > kMax31 || a.K > kMax31 || a.T > kMax31)
        return fail(TMG_ERR_UNSUPPORTED, "extents beyond 2^31");
    if (!extents_ok(a.T, a.lda, a.K, a.a_col) || !extents_ok(a.N, a.b_row, a.K, a.b_col, a.E, a.b_expert) ||
        !extents_ok(a.R, a.ldd, a.N, 1))
        return fail(TMG_ERR_INVALID_ARG, "negative strides, or offsets beyond int64");
    return TMG_OK;
}

}  // namespace

tmg_status pack(const DeviceState &ds, Workspace which, Pack3Args a, int elem, size_t total, int64_t offset, cudaStream_t s,
                char **out)
{
    tmg_status st;
    char *ws = static_cast<char *>(workspace(which, total < 16 ? 16 : total, s, &st));
    if (!ws)
        return st;
    a.dst = ws + offset;
    const cudaError_t e = launch_pack3(a, elem, ds.num_sms, s);
    if (e != cudaSuccess)
        return cuda_fail(e, "operand copy launch");
    *out = ws;
    return TMG_OK;
}

namespace {

// The tile counter and the arrival counters of split tiles, zero between
// launches.
tmg_status counters(int pairs, cudaStream_t s, uint32_t **feed, uint32_t **split)
{
    tmg_status st;
    *feed = static_cast<uint32_t *>(workspace(kWsCounters, (32 + static_cast<size_t>(pairs) * 32) * sizeof(uint32_t), s, &st));
    if (!*feed)
        return st;
    *split = *feed + 32;
    return TMG_OK;
}

// A's rows by number into workspace, rows of K elements: *A and *lda become the
// copy's.
tmg_status gather(const DeviceState &ds, const void **A, int64_t *lda, int64_t src_rows, int64_t K, int elem,
                  const int32_t *numbers, int64_t R, cudaStream_t s)
{
    const int64_t ld = up(K, 16 / elem);
    tmg_status st;
    void *ws = workspace(kWsGather, static_cast<size_t>(R) * ld * elem, s, &st);
    if (!ws)
        return st;
    const cudaError_t e = launch_gather_rows(*A, *lda * elem, src_rows, K * elem, numbers, R, ws, ld * elem, ds.num_sms, s);
    if (e != cudaSuccess)
        return cuda_fail(e, "row gather launch");
    *A = ws;
    *lda = ld;
    return TMG_OK;
}

// Nanoseconds that a CTA pair takes for one K block of a tile of w columns, over
// whole waves of tiles (measured: 256 to 8191 rows by 4096 to 14000 columns, K
// 2000 to 8192).  Narrower tiles cost more per column: every tile reads the
// weights again.
float block_ns(int w)
{
    return w <= 128 ? 245.f : w <= 160 ? 255.f : w <= 192 ? 262.f : w <= 224 ? 266.f : 295.f;
}

constexpr float kHbm = 6700.f;         // bytes a nanosecond

// HBM's time for one group's weights.
float weight_ns(const GroupedArgs &a) { return static_cast<float>(a.N) * a.K * (a.e4m3 ? 1 : 2) / kHbm; }

// Widest tile.  One group: the width whose waves of tiles take the least time
// (4096 x 4096 x 4096: 19 x 16 tiles of 224 columns are four waves of 76 pairs
// like 16 x 16 of 256, and take 79.5 us against 87; 1024 x 8192 x 8192: 82 us in
// two waves of 256 columns, 103 in three of 224).  Several: all rows of an
// evenly filled group, with room for half as many again; narrower tiles make a
// deeper ring.
int tile_width(const GroupedArgs &a, int64_t tiles_n, int64_t num_kb, int pairs)
{
    if (a.E > 1) {
        const int64_t even = (a.R + a.E - 1) / a.E, room = even + even / 2 + 8;
        return static_cast<int>(room >= kSwMaxW ? kSwMaxW : up(room, 32));
    }
    int best = 0;
    double best_ns = 0;
    for (int w = kSwMaxW; w >= 32; w -= 32) {
        SwapTail tail;
        const int64_t tiles = std::min((a.R + w - 1) / w * tiles_n, kMax31);
        const double ns = swap_time(static_cast<int>(tiles), pairs, static_cast<int>(num_kb), w, block_ns(w), weight_ns(a),
                                    tail);
        if (!best || ns < 0.95 * best_ns || (a.R <= w && ns <= best_ns)) {
            best = w;
            best_ns = ns;
        }
    }
    return best;
}

// The product over clusters: cluster 0 means the pair kernel.
struct SplitPlan {
    int cluster = 0, w = 0, tiles = 0;
};
constexpr int kSplitGatherW = 32;      // widest tile whose rows TMA gathers (8 gathers of 46 ns a K block)

// Estimated times in ns of the pair kernel and of the cluster kernel for every
// width w and cluster size S; the latter where it is expected to be faster.
// Fitted to 63 sizes (weights of 1024 .. 14000 x 1000 .. 8192, 1 to 1024 rows),
// where the choice is within 1 % of the fastest on average: the pair kernel takes
// 5.5 us + 8 w and block_ns for a K block of a tile; a wave of the cluster kernel
// 3.5 us + 27 w, 205 for a K block (320 at 256 columns) and, with S > 1, 7 w for
// the exchange; both at least what HBM (6.7 TB/s) takes for the weights and 2.8
// and 4.3 us.
SplitPlan split_plan(const GroupedArgs &a, int64_t F, bool swiglu, int64_t num_kb, int elem, int64_t pair_tiles_n, int maxw,
                     int num_sms)
{
    SplitPlan best;
    const int64_t pairs = num_sms / 2, tiles_n = (F + (swiglu ? 63 : 127)) / (swiglu ? 64 : 128);
    const int64_t groups = std::min(a.E, a.R);              // at most so many have rows
    auto row_tiles = [&](int64_t w) { return a.E == 1 ? (a.R + w - 1) / w : std::min(a.R, groups + a.R / w); };
    const double hbm = static_cast<double>(groups) * weight_ns(a);
    const int64_t pair_tiles = row_tiles(maxw) * pair_tiles_n;
    SwapTail tail;
    double best_ns = 5500 + 8 * maxw + swap_time(static_cast<int>(std::min(pair_tiles, kMax31)), static_cast<int>(pairs),
                                                 static_cast<int>(num_kb), maxw, block_ns(maxw),
                                                 static_cast<float>(hbm) + 2800, tail);
    const int64_t even = (a.R + groups - 1) / groups;
    const int64_t least = a.E == 1 ? 16 : std::min<int64_t>(256, even + even / 2 + 8);     // a group's rows in one tile
    for (int64_t w = 16; w <= 256; w *= 2) {
        const int64_t tiles = row_tiles(w) * tiles_n;
        if (w >= least && tiles <= 4 * num_sms) {
            const double gather = a.rows && w <= kSplitGatherW ? 11.5 * w : 0;
            const double block = std::max(w <= 128 ? 205.0 : 320.0, gather), fixed = 3500 + 27.0 * w;
            for (int64_t S = 1; S <= 8 && (S == 1 || num_kb >= 4 * S); S *= 2) {
                const int64_t fits = split_clusters(static_cast<int>(S));
                if (fits < 1)
                    continue;
                const double wave = fixed + (num_kb + S - 1) / S * block + (S > 1 ? 7.0 * w : 0);
                const double ns = std::max(static_cast<double>((tiles + fits - 1) / fits) * wave, hbm + 4300);
                if (ns < best_ns) {
                    best_ns = ns;
                    best.cluster = static_cast<int>(S);
                    best.w = static_cast<int>(w);
                    best.tiles = static_cast<int>(tiles);
                }
            }
        }
        if (w >= a.R)
            break;
    }
    return best;
}

}  // namespace

tmg_status run_product(const DeviceState &ds, const GroupedArgs &a, cudaStream_t s)
{
    const bool swiglu = a.epi.act == kActSwiglu;
    const int elem = a.e4m3 ? 1 : 2, align = 16 / elem, kb = a.e4m3 ? 128 : 64;
    const int64_t halves = swiglu ? 2 : 1, F = a.N / halves;
    const CUtensorMapDataType dt = a.e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    tmg_status st;
    SwapArgs p;
    std::memset(&p, 0, sizeof p);
    // the contraction that the kernel sees: an empty one is one of zeros, and
    // a copied operand's rows are padded (the other's out-of-range reads are zeros)
    const int64_t K = a.K > 0 ? a.K : align;

    const int pairs = ds.num_sms / 2;
    const int64_t tiles_n = (F + (swiglu ? 127 : 255)) / (swiglu ? 128 : 256);
    p.maxw = tile_width(a, tiles_n, (K + kb - 1) / kb, pairs);
    const SplitPlan plan = split_plan(a, F, swiglu, (K + kb - 1) / kb, elem, tiles_n, p.maxw, ds.num_sms);
    p.gather = a.rows && (plan.cluster ? plan.w <= kSplitGatherW : p.maxw <= kSwGatherW);

    // A: rows of K read in place, or copied; with row numbers and wide tiles,
    // gathered into workspace
    const void *A = a.A;
    int64_t lda = stride_or(a.T, a.lda, up(K, align)), T = a.T > 0 ? a.T : 1;
    char *ws = nullptr;
    if (!rows_in_place(A, a.T, a.lda, a.K, a.a_col, elem)) {
        lda = up(K, align);
        if ((st = pack(ds, kWsPackA, Pack3Args{A, nullptr, 1, a.T, a.K, 0, a.lda, a.a_col, T, lda, 0}, elem, T * lda * elem, 0,
                       s, &ws)) != TMG_OK)
            return st;
        A = ws;
    }
    if (a.rows && !p.gather && (st = gather(ds, &A, &lda, T, K, elem, a.rows, a.R, s)) != TMG_OK)
        return st;
    if (a.rows && !p.gather)
        T = a.R;
    // B: K-major rows, MN-major rows (plain bf16), or a K-major copy
    const void *B = a.B;
    int64_t brow = a.b_row, bexp = a.b_expert, Fp = F;
    const bool e_ok = a.E == 1 || (a.b_expert > 0 && a.b_expert * elem % 16 == 0 && a.b_expert * elem < (int64_t{1} << 40));
    bool maj = false;
    if (e_ok && (!swiglu || F % 8 == 0) && rows_in_place(B, a.N, a.b_row, a.K, a.b_col, elem)) {
        brow = stride_or(a.N, a.b_row, up(K, align));
    } else if (e_ok && !swiglu && !a.e4m3 && rows_in_place(B, a.K, a.b_col, a.N, a.b_row, elem)) {
        maj = true;
        brow = stride_or(a.K, a.b_col, up(a.N, align));
    } else {
        Fp = swiglu ? up(F, 8) : F;
        brow = up(K, align);
        bexp = halves * Fp * brow;
        for (int64_t h = 0; h < halves; ++h)
            if ((st = pack(ds, kWsPackB,
                           Pack3Args{static_cast<const char *>(a.B) + h * F * a.b_row * elem, nullptr, a.E, F, a.K, a.b_expert,
                                     a.b_row, a.b_col, Fp, brow, bexp},
                           elem, a.E * bexp * elem, h * Fp * brow * elem, s, &ws)) != TMG_OK)
                return st;
        B = ws;
    }
    bexp = stride_or(a.E, bexp, maj ? K * brow : halves * Fp * brow);

    const int64_t xdims[2] = {K, T}, xstrides[1] = {lda * elem};
    const int epi = swiglu ? kSwSwiglu : a.epi.act == kActSwigluGrad ? kSwSwigluGrad : a.offsets ? kSwPlain : kSwDense;
    if (plan.cluster) {
        SplitArgs q;
        std::memset(&q, 0, sizeof q);
        const int64_t dims[3] = {maj ? a.N : K, maj ? K : halves * Fp, a.E}, strides[2] = {brow * elem, bexp * elem};
        const int box[3] = {maj ? 64 : kb, maj || swiglu ? 64 : 128, 1}, xbox[2] = {kb, p.gather ? 1 : plan.w};
        if ((st = encode_nd(&q.tmW, dt, 3, B, dims, strides, box)) != TMG_OK ||
            (st = encode_nd(&q.tmX, dt, 2, A, xdims, xstrides, xbox)) != TMG_OK)
            return st;
        q.D = a.D;
        q.offsets = a.offsets;
        q.rows = a.rows;
        q.epi = a.epi;
        q.ldd = a.ldd;
        q.R = static_cast<int>(a.R);
        q.T = static_cast<int>(a.T);
        q.N = static_cast<int>(F);
        q.K = static_cast<int>(K);
        q.E = static_cast<int>(a.E);
        q.half_rows = static_cast<int>(Fp);
        q.maj = maj;
        q.gather = p.gather;
        q.map_rows = static_cast<int>(T);
        q.w = plan.w;
        q.tmem_cols = 32;
        while (q.tmem_cols < q.w)
            q.tmem_cols *= 2;
        q.stage_bytes = 16384 + q.w * 128;
        q.stages = 196608 / q.stage_bytes < kSplitMaxStages ? 196608 / q.stage_bytes : kSplitMaxStages;
        q.ring_bytes = q.stages * q.stage_bytes;
        log_choice("%s %s: %d rows, N=%lld K=%lld E=%d -> split_kernel: 128 x %d tiles, each over %d CTAs, weights %s%s",
                   a.e4m3 ? "e4m3" : "bf16", a.offsets ? "grouped" : "dense", q.R, (long long)a.N, (long long)a.K, q.E, q.w,
                   plan.cluster, maj ? "MN-major" : "K-major",
                   q.gather ? ", rows gathered by TMA" : a.rows ? ", rows gathered first" : "");
        return launched(launch_split(q, epi, a.e4m3, plan.cluster, plan.tiles, err_ctx(ds), s), "split product launch");
    }
    const bool reread = p.maxw > kSwGatherW;
    if (swiglu) {
        const int64_t dims[5] = {K, 8, 2, Fp / 8, a.E}, strides[4] = {brow * elem, Fp * brow * elem, 8 * brow * elem, bexp * elem};
        const int box[5] = {kb, 8, 2, 8, 1};
        st = encode_nd(&p.tmW, dt, 5, B, dims, strides, box, reread);
    } else if (maj) {
        const int64_t dims[3] = {a.N, K, a.E}, strides[2] = {brow * elem, bexp * elem};
        const int box[3] = {64, 64, 1};
        st = encode_nd(&p.tmW, dt, 3, B, dims, strides, box, reread);
    } else {
        const int64_t dims[3] = {K, a.N, a.E}, strides[2] = {brow * elem, bexp * elem};
        const int box[3] = {kb, 128, 1};
        st = encode_nd(&p.tmW, dt, 3, B, dims, strides, box, reread);
    }
    if (st != TMG_OK)
        return st;
    for (int i = 0; i < (p.gather ? 1 : 4); ++i) {
        const int box[2] = {kb, p.gather ? 1 : 16 << i};
        if ((st = encode_nd(&p.tmX[i], dt, 2, A, xdims, xstrides, box, reread)) != TMG_OK)
            return st;
    }
    p.D = a.D;
    p.offsets = a.offsets;
    p.rows = a.rows;
    p.epi = a.epi;
    p.ldd = a.ldd;
    p.R = static_cast<int>(a.R);
    p.T = static_cast<int>(a.T);
    p.map_rows = static_cast<int>(T);
    p.N = static_cast<int>(F);
    p.K = static_cast<int>(K);
    p.E = static_cast<int>(a.E);
    p.maj = maj;
    p.stage_bytes = 16384 + sw_box_rows(p.maxw / 2) * 128;
    // The dense product's results leave by TMA where their rows are 16-byte
    // aligned (5000 x 5000 x 512: 28.0 -> 26.2 us; 32 bytes a row, as SwiGLU has
    // them, gain nothing).
    auto out_map = [&](CUtensorMap *map, int *there, const void *M, int64_t ld) {
        if (epi != kSwDense || !M || !rows_in_place(M, a.R, ld, a.N, 1, 2))
            return TMG_OK;
        const int64_t dims[2] = {a.N, a.R}, strides[1] = {stride_or(a.R, ld, up(a.N, 8)) * 2};
        const int box[2] = {32, 32};
        *there = 1;
        return encode_nd(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, M, dims, strides, box);
    };
    if ((st = out_map(&p.tmD, &p.tma_d, a.D, a.ldd)) != TMG_OK ||
        (st = out_map(&p.tmP, &p.tma_p, a.epi.preact, a.epi.ld_preact)) != TMG_OK)
        return st;
    p.staging = p.tma_d || p.tma_p ? 2 * kSwStage : kSwStage;
    p.stages = kSwMaxStages;
    while (sw_smem(p.stages, p.stage_bytes, p.staging, p.E) > 232448)
        --p.stages;
    p.group = 16 * p.maxw * K * elem <= (int64_t{32} << 20) ? 16 : 8;
    if ((a.R / 32 + a.E) * tiles_n > kMax31)
        return fail(TMG_ERR_UNSUPPORTED, "more than 2^31 tiles");
    p.block_ns = block_ns(p.maxw);
    // room for the pieces of cut tiles: the kernel cuts none without.  The dense
    // product's tiles are known here, a grouped one's only there.
    const int num_kb = static_cast<int>((K + kb - 1) / kb);
    SwapTail tail{0, 1};
    if (epi == kSwDense) {
        const int total = static_cast<int>((a.R + p.maxw - 1) / p.maxw * tiles_n);
        p.hbm_ns = weight_ns(a) / total;
        swap_time(total, pairs, num_kb, p.maxw, p.block_ns, total * p.hbm_ns, tail);
    } else {
        // narrow tiles, most of them a group's only ones, read their weights once each
        p.hbm_ns = p.maxw < kSwMaxW ? 32768.f / kHbm * num_kb : 0.f;
    }
    if (epi == kSwDense ? tail.tiles > 0 : swap_may_cut(num_kb, p.maxw, p.block_ns)) {
        p.partials = static_cast<float *>(workspace(kWsPartials, pairs * sw_partial_floats(p.maxw) * sizeof(float), s, &st));
        if (!p.partials)
            return st;
    }
    if ((st = counters(pairs, s, &p.feed, &p.counters)) != TMG_OK)
        return st;
    char cuts[48] = "";
    if (tail.tiles)
        snprintf(cuts, sizeof cuts, ", %d tiles cut over %d pairs", tail.tiles, tail.tiles * tail.each);
    log_choice("%s %s: %d rows, N=%lld K=%lld E=%d -> swap_kernel: %d x up to %d tiles, %d stages, weights %s%s%s",
               a.e4m3 ? "e4m3" : "bf16", a.offsets ? "grouped" : "dense", p.R, (long long)a.N, (long long)a.K, p.E, 256, p.maxw,
               p.stages, maj ? "MN-major" : "K-major", p.gather ? ", rows gathered by TMA" : a.rows ? ", rows gathered first" : "",
               cuts);
    return launched(launch_swap(p, epi, a.e4m3, ds.num_sms, err_ctx(ds), s), "grouped product launch");
}

tmg_status run_wgrad(const DeviceState &ds, const WgradArgs &a, cudaStream_t s)
{
    tmg_status st;
    WgradTmaArgs p;
    std::memset(&p, 0, sizeof p);
    const void *op[2] = {a.dD, a.A};
    const int64_t rows[2] = {a.R, a.T}, cols[2] = {a.N, a.K}, row[2] = {a.ldd, a.lda}, col[2] = {a.d_col, a.a_col};
    for (int i = 0; i < 2; ++i) {
        int64_t ld = stride_or(rows[i], row[i], up(cols[i], 8)), n = rows[i] > 0 ? rows[i] : 1;
        if (!rows_in_place(op[i], rows[i], row[i], cols[i], col[i], 2)) {
            ld = up(cols[i], 8);
            char *ws = nullptr;
            if ((st = pack(ds, i ? kWsPackB : kWsPackA,
                           Pack3Args{op[i], nullptr, 1, rows[i], cols[i], 0, row[i], col[i], n, ld, 0}, 2, n * ld * 2, 0, s,
                           &ws)) != TMG_OK)
                return st;
            op[i] = ws;
        }
        if (i && a.rows) {
            if ((st = gather(ds, &op[i], &ld, n, cols[i], 2, a.rows, a.R, s)) != TMG_OK)
                return st;
            n = a.R;
        }
        const int64_t dims[2] = {cols[i], n}, strides[1] = {ld * 2};
        CUtensorMap *maps[3] = {i ? &p.tmA : &p.tmD, i ? &p.tmA16 : &p.tmD16, i ? &p.tmAg : &p.tmDg};
        for (int b = 0; b < 3; ++b) {
            const int box[2] = {64, b == 0 ? 64 : b == 1 ? 16 : 1};
            if ((st = encode_nd(maps[b], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, op[i], dims, strides, box, true)) != TMG_OK)
                return st;
        }
    }
    if (aligned(a.dB) && a.K % 8 == 0 && a.N * a.K * 2 < (int64_t{1} << 40)) {
        const int64_t dims[3] = {a.K, a.N, a.E}, strides[2] = {a.K * 2, a.N * a.K * 2};
        const int box[3] = {64, 32, 1};
        if ((st = encode_nd(&p.tmOut, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.dB, dims, strides, box)) != TMG_OK)
            return st;
        p.tma_out = 1;
    }
    p.dB = a.dB;
    p.offsets = a.offsets;
    p.R = static_cast<int>(a.R);
    p.N = static_cast<int>(a.N);
    p.K = static_cast<int>(a.K);
    p.E = static_cast<int>(a.E);
    p.group = 8;
    const int64_t per = ((a.N + 255) / 256) * ((a.K + 255) / 256);
    if ((a.R / 64 + 2 * a.E) * per > kMax31)
        return fail(TMG_ERR_UNSUPPORTED, "more than 2^31 tile blocks");
    const int pairs = ds.num_sms / 2;
    if ((a.R + 63) / 64 > 2 * kWgCutBlocks) {      // else no cut pays
        p.partials = static_cast<float *>(workspace(kWsPartials, wgrad_partial_bytes(ds.num_sms), s, &st));
        if (!p.partials)
            return st;
    }
    if ((st = counters(pairs, s, &p.feed, &p.counters)) != TMG_OK)
        return st;
    log_choice("bf16 grouped weight gradient: %d rows, N=%d K=%d E=%d -> wgrad_kernel: 256 x 256 tiles%s", p.R, p.N, p.K, p.E,
               a.rows ? ", rows gathered first" : "");
    return launched(launch_wgrad(p, ds.num_sms, err_ctx(ds), s), "grouped weight gradient launch");
}

}  // namespace tmg

using namespace tmg;

extern "C" {

tmg_status tmg_moe_route(const void *logits, int64_t T, int64_t E, int64_t k, int64_t ld, tmg_dtype dtype, int normalize,
                         float *weights, int32_t *experts, int32_t *offsets, int32_t *rows, int32_t *slots, void *stream)
{
    return guarded([&]() -> tmg_status {
        if (dtype != TMG_F32 && dtype != TMG_BF16)
            return fail(TMG_ERR_INVALID_ARG, "logits are fp32 or bf16 (dtype %d)", (int)dtype);
        if (T < 0 || E < 1 || E > 1024 || k < 1 || k > 16 || k > E)
            return fail(TMG_ERR_INVALID_ARG, "routing needs T >= 0, 1 <= E <= 1024 and 1 <= k <= min(16, E) (T=%lld E=%lld "
                        "k=%lld)", (long long)T, (long long)E, (long long)k);
        if (T > 1 && ld < E)
            return fail(TMG_ERR_INVALID_ARG, "row stride %lld below E=%lld", (long long)ld, (long long)E);
        if (T * k > kMax31)
            return fail(TMG_ERR_UNSUPPORTED, "T * k beyond 2^31");
        if (!offsets || (T > 0 && (!logits || !weights || !experts || !rows || !slots)))
            return fail(TMG_ERR_INVALID_ARG, "null pointer");
        DeviceState *ds = nullptr;
        tmg_status st;
        if ((st = device_state(&ds)) != TMG_OK)
            return st;
        cudaStream_t s = static_cast<cudaStream_t>(stream);
        const StreamLock lock(s);
        if (T == 0)
            return launched(cudaMemsetAsync(offsets, 0, (E + 1) * sizeof(int32_t), s), "cudaMemsetAsync(offsets)");
        RouteArgs a{};
        a.logits = logits;
        a.bf16 = dtype == TMG_BF16;
        a.T = T;
        a.ld = ld;
        a.E = static_cast<int>(E);
        a.k = static_cast<int>(k);
        a.normalize = normalize != 0;
        a.weights = weights;
        a.experts = experts;
        a.offsets = offsets;
        a.rows = rows;
        a.slots = slots;
        a.counts = static_cast<uint16_t *>(workspace(kWsRoute, route_counts_bytes(T, a.E, ds->num_sms), s, &st));
        if (!a.counts)
            return st;
        return launched(launch_route(a, ds->num_sms, s), "routing launch");
    });
}

tmg_status tmg_moe_route_backward(const void *logits, int64_t T, int64_t E, int64_t k, int64_t ld, tmg_dtype dtype,
                                  int normalize, const int32_t *experts, const float *dweights, void *dlogits,
                                  void *stream)
{
    return guarded([&]() -> tmg_status {
        if (dtype != TMG_F32 && dtype != TMG_BF16)
            return fail(TMG_ERR_INVALID_ARG, "logits are fp32 or bf16 (dtype %d)", (int)dtype);
        if (T < 0 || E < 1 || E > 1024 || k < 1 || k > 16 || k > E)
            return fail(TMG_ERR_INVALID_ARG, "routing needs T >= 0, 1 <= E <= 1024 and 1 <= k <= min(16, E) (T=%lld E=%lld "
                        "k=%lld)", (long long)T, (long long)E, (long long)k);
        if (T > 1 && ld < E)
            return fail(TMG_ERR_INVALID_ARG, "row stride %lld below E=%lld", (long long)ld, (long long)E);
        if (T == 0)
            return TMG_OK;
        if (T * k > kMax31)
            return fail(TMG_ERR_UNSUPPORTED, "T * k beyond 2^31");
        if (!logits || !experts || !dweights || !dlogits)
            return fail(TMG_ERR_INVALID_ARG, "null pointer");
        DeviceState *ds = nullptr;
        tmg_status st;
        if ((st = device_state(&ds)) != TMG_OK)
            return st;
        return launched(launch_route_backward(logits, dtype == TMG_BF16, T, ld, static_cast<int>(E), static_cast<int>(k),
                                              normalize != 0, experts, dweights, dlogits, ds->num_sms,
                                              static_cast<cudaStream_t>(stream)),
                        "routing gradient launch");
    });
}

tmg_status tmg_moe_combine(const void *Y, int64_t R, int64_t ldy, const int32_t *slots, const float *weights,
                           const void *residual, int64_t ldr, void *out, int64_t ldo, int64_t T, int64_t H, int64_t k,
                           void *stream)
{
    return guarded([&]() -> tmg_status {
        if (T < 0 || H < 0 || R < 0 || k < 1 || k > 16)
            return fail(TMG_ERR_INVALID_ARG, "combine needs T, H, R >= 0 and 1 <= k <= 16");
        if (!extents_ok(R, ldy, H, 1) || !extents_ok(T, residual ? ldr : 0, H, 1) || !extents_ok(T, ldo, H, 1) ||
            !out_rows_ok(T, H, ldo))
            return fail(TMG_ERR_INVALID_ARG, "row strides out of range (the output's must be at least H)");
        if (T == 0 || H == 0)
            return TMG_OK;
        if (T > kMax31 / 16 || H > kMax31 || T * ((H + 1023) / 1024) > kMax31)
            return fail(TMG_ERR_UNSUPPORTED, "extents beyond 2^31");
        if (!slots || !out || (R > 0 && !Y))
            return fail(TMG_ERR_INVALID_ARG, "null pointer");
        DeviceState *ds = nullptr;
        tmg_status st;
        if ((st = device_state(&ds)) != TMG_OK)
            return st;
        return launched(launch_combine(CombineArgs{Y, slots, weights, residual, out, T, H, R, ldy, ldr, ldo,
                                                   static_cast<int>(k)},
                                       static_cast<cudaStream_t>(stream)),
                        "combine launch");
    });
}

tmg_status tmg_moe_combine_backward(const void *dOut, int64_t ldo, const void *Y, int64_t R, int64_t ldy,
                                    const int32_t *slots, const float *weights, void *dY, float *dweights, int64_t T,
                                    int64_t H, int64_t k, void *stream)
{
    return guarded([&]() -> tmg_status {
        if (T < 0 || H < 0 || R < 0 || k < 1 || k > 16)
            return fail(TMG_ERR_INVALID_ARG, "combine needs T, H, R >= 0 and 1 <= k <= 16");
        if (!extents_ok(R, dweights ? ldy : 0, H, 1) || !extents_ok(T, ldo, H, 1))
            return fail(TMG_ERR_INVALID_ARG, "row strides out of range");
        if (T == 0)
            return TMG_OK;
        if (T > kMax31 / 16 || H > kMax31)
            return fail(TMG_ERR_UNSUPPORTED, "extents beyond 2^31");
        if (!slots || (H > 0 && !dOut) || (R > 0 && H > 0 && (!dY || (dweights && !Y))))
            return fail(TMG_ERR_INVALID_ARG, "null pointer");
        DeviceState *ds = nullptr;
        tmg_status st;
        if ((st = device_state(&ds)) != TMG_OK)
            return st;
        return launched(launch_combine_backward(CombineGradArgs{dOut, Y, slots, weights, dY, dweights, T, H, R, ldo, ldy,
                                                                static_cast<int>(k)},
                                                static_cast<cudaStream_t>(stream)),
                        "combine gradient launch");
    });
}

tmg_status tmg_grouped_gemm(const tmg_grouped_args *g, void *stream)
{
    return guarded([&]() -> tmg_status {
        if (!g)
            return fail(TMG_ERR_INVALID_ARG, "null argument struct");
        if (g->in_dtype == TMG_F32)
            return fail(TMG_ERR_UNSUPPORTED, "the grouped product takes bf16 or E4M3 inputs");
        if (g->in_dtype != TMG_BF16 && g->in_dtype != TMG_E4M3)
            return fail(TMG_ERR_INVALID_ARG, "unknown input dtype %d", (int)g->in_dtype);
        if (g->activation != TMG_ACT_NONE && g->activation != TMG_ACT_SWIGLU && g->activation != TMG_ACT_SWIGLU_GRAD)
            return fail(TMG_ERR_INVALID_ARG, "activation %d is not one of the grouped product's", (int)g->activation);
        if (g->E < 1 || g->E > 1024)
            return fail(TMG_ERR_INVALID_ARG, "E=%lld is not in 1 .. 1024", (long long)g->E);
        GroupedArgs a{};
        a.A = g->A;
        a.B = g->B;
        a.D = g->D;
        a.R = g->R;
        a.T = g->rows ? g->T : g->R;
        a.N = g->N;
        a.K = g->K;
        a.E = g->E;
        a.lda = g->lda;
        a.a_col = g->a_col;
        a.ldd = g->ldd;
        a.b_expert = g->b_expert;
        a.b_row = g->b_row;
        a.b_col = g->b_col;
        a.offsets = g->offsets;
        a.rows = g->rows;
        a.e4m3 = g->in_dtype == TMG_E4M3;
        a.epi.scale_a = g->scale_a;
        a.epi.scale_b = g->scale_b;
        a.epi.preact = g->activation == TMG_ACT_NONE ? nullptr : g->preact;
        a.epi.ld_preact = g->ld_preact;
        a.epi.act = g->activation;
        tmg_status st;
        if ((st = check_product(a)) != TMG_OK)
            return st;
        const bool grad = g->activation == TMG_ACT_SWIGLU_GRAD;
        if (g->activation == TMG_ACT_SWIGLU && g->N % 2)
            return fail(TMG_ERR_INVALID_ARG, "swiglu needs an even N (N=%lld)", (long long)g->N);
        const int64_t cols = grad ? 2 * g->N : g->activation == TMG_ACT_SWIGLU ? g->N / 2 : g->N;
        if (!out_rows_ok(g->R, cols, g->ldd))
            return fail(TMG_ERR_INVALID_ARG, "row stride %lld of D below its %lld columns", (long long)g->ldd,
                        (long long)cols);
        if (grad && !g->preact && g->R > 0 && g->N > 0)
            return fail(TMG_ERR_INVALID_ARG, "swiglu_grad reads preact, which is NULL");
        if (a.epi.preact && (g->ld_preact < 0 || !out_rows_ok(g->R, grad ? 2 * g->N : g->N, g->ld_preact)))
            return fail(TMG_ERR_INVALID_ARG, "row stride %lld of preact too small", (long long)g->ld_preact);
        if (g->R == 0 || g->N == 0)
            return TMG_OK;
        if (!g->offsets || !g->D || (g->K > 0 && (!g->B || (a.T > 0 && !g->A))))
            return fail(TMG_ERR_INVALID_ARG, "null pointer");
        DeviceState *ds = nullptr;
        if ((st = device_state(&ds)) != TMG_OK)
            return st;
        const StreamLock lock(static_cast<cudaStream_t>(stream));
        return run_product(*ds, a, static_cast<cudaStream_t>(stream));
    });
}

tmg_status tmg_grouped_gemm_wgrad(const void *dD, int64_t ldd, int64_t d_col, const void *A, int64_t lda, int64_t a_col,
                                  void *dB, const int32_t *offsets, const int32_t *rows, int64_t R, int64_t N, int64_t K,
                                  int64_t E, int64_t T, void *stream)
{
    return guarded([&]() -> tmg_status {
        if (R < 0 || N < 0 || K < 0 || T < 0)
            return fail(TMG_ERR_INVALID_ARG, "negative extent R=%lld N=%lld K=%lld T=%lld", (long long)R, (long long)N,
                        (long long)K, (long long)T);
        if (E < 1 || E > 1024)
            return fail(TMG_ERR_INVALID_ARG, "E=%lld is not in 1 .. 1024", (long long)E);
        if (R > kMax31 || N > kMax31 || K > kMax31 || T > kMax31)
            return fail(TMG_ERR_UNSUPPORTED, "extents beyond 2^31");
        if (!rows)
            T = R;
        if (!extents_ok(R, ldd, N, d_col) || !extents_ok(T, lda, K, a_col))
            return fail(TMG_ERR_INVALID_ARG, "negative strides, or offsets beyond int64");
        if (N == 0 || K == 0)
            return TMG_OK;
        if (!dB || !offsets || (R > 0 && !dD) || (T > 0 && R > 0 && !A))
            return fail(TMG_ERR_INVALID_ARG, "null pointer");
        DeviceState *ds = nullptr;
        tmg_status st;
        if ((st = device_state(&ds)) != TMG_OK)
            return st;
        const cudaStream_t s = static_cast<cudaStream_t>(stream);
        const StreamLock lock(s);
        if (R == 0)                    // the kernel's operand maps have a row at least
            return launched(cudaMemsetAsync(dB, 0, static_cast<size_t>(E) * N * K * 2, s), "cudaMemsetAsync(dB)");
        return run_wgrad(*ds, WgradArgs{dD, A, dB, R, T, N, K, E, ldd, d_col, lda, a_col, offsets, rows}, s);
    });
}

tmg_status tmg_linear(const tmg_linear_args *g, void *stream)
{
    return guarded([&]() -> tmg_status {
        if (!g)
            return fail(TMG_ERR_INVALID_ARG, "null argument struct");
        if (g->in_dtype == TMG_F32)
            return fail(TMG_ERR_UNSUPPORTED, "the dense product with the residual epilogue takes bf16 or E4M3 inputs");
        if (g->in_dtype != TMG_BF16 && g->in_dtype != TMG_E4M3)
            return fail(TMG_ERR_INVALID_ARG, "unknown input dtype %d", (int)g->in_dtype);
        if (g->activation < TMG_ACT_NONE || g->activation > TMG_ACT_GELU)
            return fail(TMG_ERR_INVALID_ARG, "activation %d is not one of the dense product's", (int)g->activation);
        GroupedArgs a{};
        a.A = g->A;
        a.B = g->B;
        a.D = g->D;
        a.R = a.T = g->M;
        a.N = g->N;
        a.K = g->K;
        a.E = 1;
        a.lda = g->lda;
        a.a_col = g->a_col;
        a.ldd = g->ldd;
        a.b_row = g->b_row;
        a.b_col = g->b_col;
        a.e4m3 = g->in_dtype == TMG_E4M3;
        a.epi = ProductEpi{g->scale_a, g->scale_b, g->bias, g->residual, g->preact, g->ld_residual, g->ld_preact,
                           static_cast<int>(g->activation)};
        tmg_status st;
        if ((st = check_product(a)) != TMG_OK)
            return st;
        if (!out_rows_ok(g->M, g->N, g->ldd) || (g->preact && !out_rows_ok(g->M, g->N, g->ld_preact)) ||
            (g->residual && !extents_ok(g->M, g->ld_residual, g->N, 1)))
            return fail(TMG_ERR_INVALID_ARG, "row stride of D, preact or residual out of range");
        if (g->M == 0 || g->N == 0)
            return TMG_OK;
        if (!g->D || (g->K > 0 && (!g->A || !g->B)))
            return fail(TMG_ERR_INVALID_ARG, "null pointer");
        DeviceState *ds = nullptr;
        if ((st = device_state(&ds)) != TMG_OK)
            return st;
        const StreamLock lock(static_cast<cudaStream_t>(stream));
        return run_product(*ds, a, static_cast<cudaStream_t>(stream));
    });
}

tmg_status tmg_linear_backward(const void *dD, int64_t ldd, const void *preact, int64_t ldp, const void *A, int64_t lda,
                               const void *B, int64_t ldb, void *dA, void *dB, float *dbias, int64_t M, int64_t N,
                               int64_t K, tmg_activation activation, void *stream)
{
    return guarded([&]() -> tmg_status {
        if (activation < TMG_ACT_NONE || activation > TMG_ACT_GELU)
            return fail(TMG_ERR_INVALID_ARG, "activation %d is not one of the dense product's", (int)activation);
        if (M < 0 || N < 0 || K < 0)
            return fail(TMG_ERR_INVALID_ARG, "negative extent M=%lld N=%lld K=%lld", (long long)M, (long long)N,
                        (long long)K);
        if (M > kMax31 || N > kMax31 || K > kMax31)
            return fail(TMG_ERR_UNSUPPORTED, "extents beyond 2^31");
        const bool act = activation != TMG_ACT_NONE;
        if (!extents_ok(M, ldd, N, 1) || !extents_ok(M, act ? ldp : 0, N, 1) || !extents_ok(M, lda, K, 1) ||
            !extents_ok(N, ldb, K, 1))
            return fail(TMG_ERR_INVALID_ARG, "negative strides, or offsets beyond int64");
        if (M > 0 && N > 0 && (!dD || (act && !preact)))
            return fail(TMG_ERR_INVALID_ARG, "null pointer (dD, or the preact that the activation's gradient reads)");
        if ((dA && K > 0 && N > 0 && !B) || (dB && K > 0 && M > 0 && !A))
            return fail(TMG_ERR_INVALID_ARG, "null pointer: dA needs B, dB needs A");
        DeviceState *ds = nullptr;
        tmg_status st;
        if ((st = device_state(&ds)) != TMG_OK)
            return st;
        cudaStream_t s = static_cast<cudaStream_t>(stream);
        const StreamLock lock(s);
        const void *dz = dD;
        int64_t ldz = ldd;
        if (M > 0 && N > 0 && (act || dbias)) {
            const size_t part = static_cast<size_t>(act_grad_chunks(M, N)) * N * sizeof(float);
            const size_t grad = act ? static_cast<size_t>(M) * N * 2 : 0;
            char *ws = static_cast<char *>(workspace(kWsGrad, (part + 255) / 256 * 256 + grad, s, &st));
            if (!ws)
                return st;
            void *z = act ? ws + (part + 255) / 256 * 256 : nullptr;
            if ((st = launched(launch_act_grad(dD, ldd, preact, ldp, activation, M, N, z, reinterpret_cast<float *>(ws),
                                               dbias, s),
                               "activation gradient launch")) != TMG_OK)
                return st;
            if (act) {
                dz = z;
                ldz = N;
            }
        } else if (dbias && N > 0) {
            if ((st = launched(cudaMemsetAsync(dbias, 0, N * sizeof(float), s), "cudaMemsetAsync(dbias)")) != TMG_OK)
                return st;
        }
        // dA (M, K) = dz (M, N) . B: B read as (K, N); dB (N, K) = dz^T . A.  Each
        // by the kernel that is faster.  Where the tiles do not fill the CTA pairs, or
        // there are less than 256 rows, the GEMM would copy the MN-major operands (165
        // x 6408 x 736: dA 35 us against 12 with the dense product; 250 x 4096 x 24576:
        // all 196 against 116; 2795 x 624 x 4024: dB 30 against 22 with the weight
        // gradient; one row of 4096 x 4096: dB 73 against 15).
        // Where they do, its pair kernel reads them in place and is faster on short
        // contractions (8191 x 4096 x 4096: dA 144 against 148; 1024 x 4096 x 4096:
        // dB 26 against 30), slower on long ones (2048 x 8192 x 8192: dA 164 against
        // 150; 6080 x 4520 x 3400: 151 against 144, dB 156 against 146; 8191 x 4096
        // x 4096: dB 165 against 159) and where rows begin inside a sector (2833 x
        // 6648 x 6800: dA 183 against 161, dB 169 against 161; 74 x 7016 x 6296: dB
        // 36 against 29).
        auto fills = [&](int64_t rows, int64_t cols) {
            return rows >= 256 && (rows + 255) / 256 * ((cols + 255) / 256) >= ds->num_sms / 2;
        };
        const bool some = M > 0 && N > 0 && K > 0;
        const bool a_product = some && (!fills(M, K) || N > 4096 || (ldz | ldb) % 16);
        const bool b_wgrad = some && (!fills(N, K) || M < 64 || (M > 6000 && M >= N && M >= K) || (ldz | lda) % 16);
        auto flat = [](int64_t r, int64_t c, int64_t sr, int64_t sc) {
            tmg_layout L;
            std::memset(&L, 0, sizeof L);
            L.depth[0] = L.depth[1] = 1;
            L.shape[0][0] = r;
            L.shape[1][0] = c;
            L.shape[0][1] = L.shape[1][1] = 1;
            L.stride[0][0] = sr;
            L.stride[1][0] = sc;
            return L;
        };
        if (dA && a_product) {
            GroupedArgs a{};
            a.A = dz;
            a.B = B;
            a.D = dA;
            a.R = a.T = M;
            a.N = a.ldd = K;
            a.K = N;
            a.E = 1;
            a.lda = ldz;
            a.a_col = a.b_row = 1;
            a.b_col = ldb;
            if ((st = run_product(*ds, a, s)) != TMG_OK)
                return st;
        } else if (dA) {
            const tmg_layout lz = flat(M, N, ldz, 1), lb = flat(K, N, 1, ldb);
            if ((st = tmg_gemm_ex(dz, B, dA, M, K, N, TMG_BF16, &lz, &lb, nullptr, TMG_PATH_AUTO, stream)) != TMG_OK)
                return st;
        }
        if (dB && b_wgrad) {
            if ((st = run_wgrad(*ds, WgradArgs{dz, A, dB, M, M, N, K, 1, ldz, 1, lda, 1, nullptr, nullptr}, s)) != TMG_OK)
                return st;
        } else if (dB) {
            const tmg_layout lz = flat(N, M, 1, ldz), la = flat(K, M, 1, lda);
            if ((st = tmg_gemm_ex(dz, A, dB, N, K, M, TMG_BF16, &lz, &la, nullptr, TMG_PATH_AUTO, stream)) != TMG_OK)
                return st;
        }
        return TMG_OK;
    });
}

}  // extern "C"
