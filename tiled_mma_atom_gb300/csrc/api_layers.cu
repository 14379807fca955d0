// api_layers.cu — C ABI of the calls that run several products: the whole expert
// layer, and the dense product with low-rank adapters (include/tmg.h).
#include <algorithm>
#include <cstring>

#include "act.cuh"
#include "lora.h"
#include "moe_few.h"
#include "product.h"
#include "swap_kernel.cuh"

namespace tmg {
namespace {

// Pieces of one workspace, 256-byte aligned.
struct Pieces {
    size_t bytes = 0;
    size_t take(size_t n)
    {
        const size_t at = bytes;
        bytes += (n + 255) / 256 * 256;
        return at;
    }
};

// Arrival counters, zero between launches (the tile feed's counter comes before
// them).
tmg_status arrival_counters(size_t n, cudaStream_t s, uint32_t **out)
{
    tmg_status st;
    *out = static_cast<uint32_t *>(workspace(kWsCounters, (32 + n) * sizeof(uint32_t), s, &st));
    if (*out)
        *out += 32;
    return st;
}

// The layer by the separate operators: plan, up products, down products, sum.
tmg_status moe_by_groups(const DeviceState &ds, const tmg_moe_args &g, cudaStream_t s)
{
    tmg_status st;
    const int64_t R = g.T * g.k;
    Pieces p;
    const size_t weights = p.take(R * 4), experts = p.take(R * 4), offsets = p.take((g.E + 1) * 4), rows = p.take(R * 4),
                 slots = p.take(R * 4), hidden = p.take(R * up(g.F, 8) * 2), answers = p.take(R * up(g.H, 8) * 2);
    char *ws = static_cast<char *>(workspace(kWsLayer, p.bytes, s, &st));
    if (!ws)
        return st;
    RouteArgs r{};
    r.logits = g.logits;
    r.bf16 = g.logits_dtype == TMG_BF16;
    r.T = g.T;
    r.ld = g.ld_logits;
    r.E = static_cast<int>(g.E);
    r.k = static_cast<int>(g.k);
    r.normalize = g.normalize != 0;
    r.weights = reinterpret_cast<float *>(ws + weights);
    r.experts = reinterpret_cast<int32_t *>(ws + experts);
    r.offsets = reinterpret_cast<int32_t *>(ws + offsets);
    r.rows = reinterpret_cast<int32_t *>(ws + rows);
    r.slots = reinterpret_cast<int32_t *>(ws + slots);
    r.counts = static_cast<uint16_t *>(workspace(kWsRoute, route_counts_bytes(g.T, r.E, ds.num_sms), s, &st));
    if (!r.counts)
        return st;
    if ((st = launched(launch_route(r, ds.num_sms, s), "routing launch")) != TMG_OK)
        return st;
    GroupedArgs a{};
    a.R = R;
    a.E = g.E;
    a.b_col = a.a_col = 1;
    a.offsets = r.offsets;
    if (g.F > 0) {
        a.A = g.x;
        a.B = g.W1;
        a.D = ws + hidden;
        a.T = g.T;
        a.N = 2 * g.F;
        a.K = a.b_row = g.H;
        a.lda = g.ldx;
        a.ldd = up(g.F, 8);
        a.b_expert = 2 * g.F * g.H;
        a.rows = r.rows;
        a.epi.act = kActSwiglu;
        if ((st = run_product(ds, a, s)) != TMG_OK)
            return st;
    }
    a.A = ws + hidden;
    a.B = g.W2;
    a.D = ws + answers;
    a.T = R;
    a.N = g.H;
    a.K = a.b_row = g.F;
    a.lda = up(g.F, 8);
    a.ldd = up(g.H, 8);
    a.b_expert = g.H * g.F;
    a.rows = nullptr;
    a.epi.act = kActNone;
    if ((st = run_product(ds, a, s)) != TMG_OK)
        return st;
    return launched(launch_combine(CombineArgs{a.D, r.slots, r.weights, g.residual, g.out, g.T, g.H, R, a.ldd, g.ld_residual,
                                               g.ld_out, r.k},
                                   s),
                    "combine launch");
}

// Rows of `cols` elements that TMA can read: in place, or copied to workspace `which`
// (rows_p rows, the ones past `rows` zeros).
struct Rows {
    const void *p;
    int64_t ld;
};
tmg_status tma_rows(const DeviceState &ds, Workspace which, const void *src, int64_t ld, int64_t rows, int64_t cols,
                    int64_t rows_p, cudaStream_t s, Rows *out)
{
    const int64_t least = up(std::max<int64_t>(cols, 1), 8);
    // a single row's end is not padded, and some kernels read whole 16 bytes
    if (rows_in_place(src, rows, ld, cols, 1, 2) && (rows > 1 || cols % 8 == 0)) {
        *out = Rows{src, stride_or(rows, ld, least)};
        return TMG_OK;
    }
    char *ws = nullptr;
    const tmg_status st = pack(ds, which, Pack3Args{src, nullptr, 1, rows, cols, 0, ld, 1, rows_p, least, 0}, 2,
                               rows_p * least * 2, 0, s, &ws);
    *out = Rows{ws, least};
    return st;
}

// One side of the factors' gradients: G from Y (M, C) and Z (M, r).
tmg_status grad_side(LoraGradSide &g, const Rows &Y, int64_t C, const Rows &Z, int64_t M, void *G, bool across)
{
    tmg_status st;
    for (int i = 0; i < 3; ++i) {
        const int64_t dims[2] = {C, M}, strides[1] = {Y.ld * 2};
        const int box[2] = {64, i == 0 ? 64 : i == 1 ? 16 : 1};
        if ((st = encode_nd(&g.tmY[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, Y.p, dims, strides, box)) != TMG_OK)
            return st;
    }
    g.Z = Z.p;
    g.ldz = Z.ld;
    g.G = G;
    g.C = static_cast<int>(C);
    g.across = across;
    return TMG_OK;
}

tmg_status run_grad(const DeviceState &ds, LoraGradArgs &p, cudaStream_t s)
{
    tmg_status st;
    p.partials = static_cast<float *>(workspace(kWsPartials, lora_grad_partial_bytes(p, ds.num_sms), s, &st));
    if (!p.partials || (st = arrival_counters(lora_grad_counters(p, ds.num_sms), s, &p.counters)) != TMG_OK)
        return st;
    return launched(launch_lora_grad(p, ds.num_sms, err_ctx(ds), s), "adapter gradient launch");
}

// A few rows' ranks: a warp per row and rank, where 16-byte loads read the factors in
// place.  With more rows the tensor cores' way is faster (65 x 4096 x 4096 18.7 us
// against 19.4 in all, 100 18.0 and 21.5; 60 rows of rank 64 38.0 and 18.7).
bool few_ranks(const RankArgs &a)
{
    return a.M <= kLoraFewRows && a.r <= kLoraFewRanks && !a.across && a.C % 8 == 0 && aligned(a.F);
}

// U = bf16(scales X . F[adapters]^T), (M, r) with rows of ldu; x, f: X's and F's rows
// as tma_rows gave them, f only where few_ranks() does not hold.  beside: the kernel
// before is launch_lora_plan's.
tmg_status run_rank(const DeviceState &ds, const RankArgs &a, const Rows &x, const Rows &f, bool beside, cudaStream_t s)
{
    if (a.C == 0)
        return launched(cudaMemsetAsync(a.U, 0, static_cast<size_t>(a.M) * a.ldu * 2, s), "cudaMemsetAsync(u)");
    if (few_ranks(a)) {
        RankArgs b = a;
        b.X = x.p;
        b.ldx = x.ld;
        return launched(launch_lora_few_rank(b, ds.num_sms, s), "adapter rank launch");
    }
    tmg_status st;
    const int64_t rows = a.across ? a.C : a.r, cols = a.across ? a.r : a.C;
    LoraRankArgs p;
    std::memset(&p, 0, sizeof p);
    const CUtensorMapDataType bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const int64_t xd[2] = {a.C, a.M}, xs[1] = {x.ld * 2}, fd[3] = {cols, rows, a.L}, fs[2] = {f.ld * 2, rows * f.ld * 2};
    const int xbox[2] = {64, 128}, fbox[3] = {64, a.across ? 64 : (a.r + 15) & ~15, 1};
    if ((st = encode_nd(&p.tmX, bf16, 2, x.p, xd, xs, xbox)) != TMG_OK ||
        (st = encode_nd(&p.tmF, bf16, 3, f.p, fd, fs, fbox, true)) != TMG_OK)
        return st;
    p.adapters = a.adapters;
    p.scales = a.scales;
    p.U = a.U;
    p.ldu = a.ldu;
    p.M = static_cast<int>(a.M);
    p.C = static_cast<int>(a.C);
    p.L = static_cast<int>(a.L);
    p.r = a.r;
    p.beside = beside;
    return launched(launch_lora_rank_tc(p, a.across, ds.num_sms, err_ctx(ds), s), "adapter rank launch");
}

// D = x . W^T + U . F[adapters]^T + bias + residual.  The factors' own strides are
// their contiguous ones; across: W is (K, N), F (L, r, N), as the input's gradient has
// them.
struct AdaptedArgs {
    Rows x, W, F;              // as tma_rows gave them, before the kernel that makes U
    const void *U;
    void *D;
    const int32_t *adapters;
    const float *bias;
    const void *residual;
    int64_t M, N, K, r, L;
    int64_t ldu, ldd, ld_residual;
    bool across;
};

// The CTAs that share a tile of 128 x 128 (lora_split.cu), or 0 for the pair kernel.
// Where such tiles are at most one for two SMs and the contraction is long, splitting
// it beats the pairs' larger tiles (100 x 4096 x 4096 17.6 us against 20.0, 128 x 8192 x
// 8192 33.4 and 46.7, 700 x 1024 x 4096 16.1 and 20.5); with more tiles or a short one it
// does not (400 x 4096 x 4096 28.4 and 26.6, 1000 x 1024 x 1024 13.1 and 10.1).
int split_cluster(int64_t M, int64_t N, int num_kb, int num_sms)
{
    const int64_t tiles = (M + 127) / 128 * ((N + 127) / 128);
    if (2 * tiles > num_sms || num_kb < 32)
        return 0;
    int S = 2;
    while (S < 8 && 2 * S * tiles <= num_sms && num_kb >= 8 * S)
        S *= 2;
    return S;
}

// Kernel and tiles of a product with adapters.
struct AdaptedTiles {
    int split;                 // split_cluster()'s
    int bn;                    // the tile's width, and the cut of the last wave, of the pair kernel
    SwapTail tail;
    int64_t ctas;              // one per SM, or two of the cluster kernel's
};

// The pair kernel's tile width and cut: the least time of the waves, a K block of a tile
// taking as long as in the GEMM's pair kernel.
tmg_status adapted_tiles(const AdaptedArgs &a, int num_sms, AdaptedTiles *t)
{
    const int pairs = num_sms / 2, num_kb = static_cast<int>((std::max<int64_t>(a.K, 1) + 63) / 64);
    *t = AdaptedTiles{split_cluster(a.M, a.N, num_kb, num_sms), 256, SwapTail{0, 1}, 0};
    if (t->split) {                            // boxes of 128 rows, as of the widest tile
        t->ctas = t->split * ((a.M + 127) / 128) * ((a.N + 127) / 128);
        return TMG_OK;
    }
    float best = 0.f;
    for (int w : {256, 224, 192, 128}) {
        if (a.across && w != 256 && w != 128)
            continue;                          // boxes of 64 columns for each CTA of the pair
        const int64_t tiles = (a.M + 255) / 256 * ((a.N + w - 1) / w);
        if (tiles > kMax31)
            return fail(TMG_ERR_UNSUPPORTED, "more than 2^31 tiles");
        SwapTail tail;
        const float ns = swap_time(static_cast<int>(tiles), pairs, num_kb, w, w == 256 ? 320.f : w == 224 ? 281.f : w == 192 ? 244.f : 204.f,
                                   0.f, tail);
        if (w == 256 || ns < best) {
            *t = AdaptedTiles{0, w, tail, tail.tiles > 0 ? 2 * pairs : 2 * std::min<int64_t>(tiles, pairs)};
            best = ns;
        }
    }
    return TMG_OK;
}

tmg_status run_adapted(const DeviceState &ds, const AdaptedArgs &a, const AdaptedTiles &t, cudaStream_t s)
{
    tmg_status st;
    LoraPairArgs p;
    std::memset(&p, 0, sizeof p);
    const CUtensorMapDataType bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const int64_t K = a.K > 0 ? a.K : 8;       // an empty contraction is one of zeros
    const int pairs = ds.num_sms / 2, bn = t.bn;
    const int64_t frows = a.across ? a.r : a.N, fcols = a.across ? a.N : a.r;
    const int64_t xd[2] = {K, a.M}, xs[1] = {a.x.ld * 2}, ud[2] = {a.r, a.M}, us[1] = {a.ldu * 2};
    const int rows[2] = {64, 128}, half[3] = {64, a.across ? 64 : bn / 2, 1};
    const int64_t wd[2] = {a.across ? a.N : K, a.across ? K : a.N}, wst[1] = {a.W.ld * 2};
    const int64_t fd[3] = {fcols, frows, a.L}, fs[2] = {a.F.ld * 2, frows * a.F.ld * 2};
    if ((st = encode_nd(&p.tmX, bf16, 2, a.x.p, xd, xs, rows, true)) != TMG_OK ||
        (st = encode_nd(&p.tmU, bf16, 2, a.U, ud, us, rows, true)) != TMG_OK ||
        (st = encode_nd(&p.tmW, bf16, 2, a.W.p, wd, wst, half, true)) != TMG_OK ||
        (st = encode_nd(&p.tmF, bf16, 3, a.F.p, fd, fs, half, true)) != TMG_OK)
        return st;
    p.M = static_cast<int>(a.M);
    p.N = static_cast<int>(a.N);
    p.K = static_cast<int>(K);
    if (t.split) {
        p.D = a.D;
        p.adapters = a.adapters;
        p.bias = a.bias;
        p.residual = a.residual;
        p.ldd = a.ldd;
        p.ld_residual = a.ld_residual;
        p.L = static_cast<int>(a.L);
        p.r = static_cast<int>(a.r);
        return launched(launch_lora_split(p, a.across, t.split, err_ctx(ds), s), "product with adapters launch");
    }
    p.group_m = 16 * 256 * static_cast<int64_t>(K) * 2 <= (int64_t{32} << 20) ? 16 : 8;
    p.cut_tiles = t.tail.tiles;
    p.cut_pieces = t.tail.each;
    if (t.tail.tiles > 0) {
        p.partials = static_cast<float *>(workspace(kWsTc2Partials, pairs * sw_partial_floats(bn) * sizeof(float), s, &st));
        if (!p.partials)
            return st;
    }
    // counters apart from those of the adapters' gradients, beside which this kernel may run
    p.feed = static_cast<uint32_t *>(workspace(kWsTc2Counters, (32 + static_cast<size_t>(pairs) * 16) * sizeof(uint32_t), s, &st));
    if (!p.feed)
        return st;
    p.counters = p.feed + 32;
    p.D = a.D;
    p.adapters = a.adapters;
    p.bias = a.bias;
    p.residual = a.residual;
    p.ldd = a.ldd;
    p.ld_residual = a.ld_residual;
    p.L = static_cast<int>(a.L);
    p.r = static_cast<int>(a.r);
    p.vec_ok = a.ldd % 8 == 0 && aligned(a.D);
    log_choice("bf16 with adapters: %d rows, N=%d K=%d rank %d -> lora_pair_kernel: 256 x %d tiles, weights %s, %d tiles cut over %d pairs",
               p.M, p.N, p.K, p.r, bn, a.across ? "MN-major" : "K-major", t.tail.tiles, t.tail.tiles * t.tail.each);
    return launched(launch_lora_pair(p, bn, a.across, static_cast<int>(t.ctas / 2), err_ctx(ds), s), "product with adapters launch");
}

// The layer in two kernels (three with more than 16 tokens), for few tokens: 16 tokens of
// 64 experts, 2048 x 1024, 119 us against 131 by groups, 13 of 32 experts, 4096 x 2048, 171
// and 184, 61 of 64 experts, 2048 x 1024, 143 and 145, one token 26 and 33; with one rounding between the products where the groups
// have two.
bool few_tokens(const tmg_moe_args &g)
{
    return g.T <= kFewTokens && g.E <= kFewExperts && g.H % 8 == 0 && g.F % 8 == 0 && g.F > 0 && aligned(g.W1) && aligned(g.W2) &&
           rows_in_place(g.x, g.T, g.ldx, g.H, 1, 2) && g.F * g.H * 4 < (int64_t{1} << 40) && g.F <= kMax31 / 4;
}

tmg_status moe_few(const DeviceState &ds, const tmg_moe_args &g, cudaStream_t s)
{
    tmg_status st;
    MoeFewArgs p;
    std::memset(&p, 0, sizeof p);
    const CUtensorMapDataType bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const int64_t experts = std::min(g.E, g.T * g.k), tp = up(g.T, 16);
    Pieces w;
    const size_t hidden = w.take(experts * tp * g.F * 2), weights = w.take(g.T * g.k * 4), chosen = w.take(g.T * g.k * 4);
    char *ws = static_cast<char *>(workspace(kWsLayer, w.bytes, s, &st));
    if (!ws)
        return st;
    p.hidden = ws + hidden;
    p.weights = reinterpret_cast<float *>(ws + weights);
    p.chosen = reinterpret_cast<int32_t *>(ws + chosen);
    const int64_t d1[3] = {g.H, 2 * g.F, g.E}, s1[2] = {g.H * 2, g.F * g.H * 4};
    const int64_t d2[3] = {g.F, g.H, g.E}, s2[2] = {g.F * 2, g.F * g.H * 2};
    const int64_t dx[2] = {g.H, g.T}, sx[1] = {stride_or(g.T, g.ldx, g.H) * 2};
    const int64_t dh[3] = {g.F, tp, experts}, sh[2] = {g.F * 2, tp * g.F * 2};
    const int b1[3] = {64, 64, 1}, b2[3] = {64, 128, 1}, bt[3] = {64, static_cast<int>(tp), 1};
    if ((st = encode_nd(&p.tmW1, bf16, 3, g.W1, d1, s1, b1)) != TMG_OK || (st = encode_nd(&p.tmW2, bf16, 3, g.W2, d2, s2, b2)) != TMG_OK ||
        (st = encode_nd(&p.tmX, bf16, 2, g.x, dx, sx, bt, true)) != TMG_OK ||
        (st = encode_nd(&p.tmHidden, bf16, 3, p.hidden, dh, sh, bt, true)) != TMG_OK)
        return st;
    p.logits = g.logits;
    p.W2 = g.W2;
    p.residual = g.residual;
    p.out = g.out;
    p.ld_logits = g.ld_logits;
    p.ld_residual = g.ld_residual;
    p.ld_out = g.ld_out;
    p.T = static_cast<int>(g.T);
    p.H = static_cast<int>(g.H);
    p.F = static_cast<int>(g.F);
    p.E = static_cast<int>(g.E);
    p.k = static_cast<int>(g.k);
    p.normalize = g.normalize != 0;
    p.bf16 = g.logits_dtype == TMG_BF16;
    p.shape.tp = static_cast<int>(tp);
    return launched(launch_moe_few(p, ds.num_sms, err_ctx(ds), s), "expert layer launch");
}

// The same for a few rows, not across; with: U by the same kernel, to with->U if that is
// not null.
tmg_status run_adapted_few(const DeviceState &ds, const AdaptedArgs &a, const RankArgs *with, cudaStream_t s)
{
    tmg_status st;
    LoraFewArgs p;
    std::memset(&p, 0, sizeof p);
    const int64_t K = a.K > 0 ? a.K : 8, tp = up(a.M, 16);
    const int64_t wd[2] = {K, a.N}, wst[1] = {a.W.ld * 2}, xd[2] = {K, a.M}, xs[1] = {a.x.ld * 2};
    const int wbox[2] = {64, 128}, xbox[2] = {64, static_cast<int>(tp)};
    if ((st = encode_nd(&p.tmW, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.W.p, wd, wst, wbox)) != TMG_OK ||
        (st = encode_nd(&p.tmX, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.x.p, xd, xs, xbox, true)) != TMG_OK)
        return st;
    if (with) {
        p.U = with->U;
        p.X = a.x.p;
        p.ldx = a.x.ld;
        p.A = with->F;
        p.scales = with->scales;
    } else {
        p.U = const_cast<void *>(a.U);
    }
    p.F = a.F.p;
    p.D = a.D;
    p.adapters = a.adapters;
    p.bias = a.bias;
    p.residual = a.residual;
    p.ldu = a.ldu;
    p.ldf = a.F.ld;
    p.ldd = a.ldd;
    p.ld_residual = a.ld_residual;
    p.M = static_cast<int>(a.M);
    p.N = static_cast<int>(a.N);
    p.K = static_cast<int>(K);
    p.L = static_cast<int>(a.L);
    p.r = static_cast<int>(a.r);
    p.shape.tp = static_cast<int>(tp);
    return launched(launch_lora_few(p, ds.num_sms, err_ctx(ds), s), "product with adapters launch");
}

// Limits of the adapters' extents and pointers, common to both directions.
tmg_status check_lora(int64_t M, int64_t N, int64_t K, int64_t r, int64_t L)
{
    if (M < 0 || N < 0 || K < 0 || r < 1 || r > 256 || L < 1 || L > 1024)
        return fail(TMG_ERR_INVALID_ARG, "adapters need M, N, K >= 0, 1 <= rank <= 256 and 1 <= L <= 1024 (M=%lld N=%lld K=%lld "
                    "rank=%lld L=%lld)", (long long)M, (long long)N, (long long)K, (long long)r, (long long)L);
    const int64_t most = kMax31 - 1024;          // a tile past the last row or column is still an int
    if (M > most || N > most || K > most)
        return fail(TMG_ERR_UNSUPPORTED, "extents beyond 2^31 - 1024");
    return TMG_OK;
}

}  // namespace
}  // namespace tmg

using namespace tmg;

extern "C" {

tmg_status tmg_moe_layer(const tmg_moe_args *g, void *stream)
{
    return guarded([&]() -> tmg_status {
        if (!g)
            return fail(TMG_ERR_INVALID_ARG, "null argument struct");
        if (g->logits_dtype != TMG_F32 && g->logits_dtype != TMG_BF16)
            return fail(TMG_ERR_INVALID_ARG, "logits are fp32 or bf16 (dtype %d)", (int)g->logits_dtype);
        if (g->T < 0 || g->H < 0 || g->F < 0 || g->E < 1 || g->E > 1024 || g->k < 1 || g->k > 16 || g->k > g->E)
            return fail(TMG_ERR_INVALID_ARG, "the expert layer needs T, H, F >= 0, 1 <= E <= 1024 and 1 <= k <= min(16, E) "
                        "(T=%lld H=%lld F=%lld E=%lld k=%lld)", (long long)g->T, (long long)g->H, (long long)g->F,
                        (long long)g->E, (long long)g->k);
        if (g->T > kMax31 / 16 || g->H > kMax31 || g->F > kMax31 / 2 || g->T * ((g->H + 1023) / 1024) > kMax31)
            return fail(TMG_ERR_UNSUPPORTED, "extents beyond 2^31");
        if (g->T > 1 && g->ld_logits < g->E)
            return fail(TMG_ERR_INVALID_ARG, "row stride %lld of the logits below E=%lld", (long long)g->ld_logits,
                        (long long)g->E);
        if (!extents_ok(g->T, g->ldx, g->H, 1) || !extents_ok(g->T, g->residual ? g->ld_residual : 0, g->H, 1) ||
            !extents_ok(g->T, g->ld_out, g->H, 1) || !out_rows_ok(g->T, g->H, g->ld_out) ||
            static_cast<__int128>(g->E) * 2 * g->F * g->H >= static_cast<__int128>(1) << 60)
            return fail(TMG_ERR_INVALID_ARG, "row strides out of range (the output's must be at least H), or weights beyond int64");
        if (g->T == 0 || g->H == 0)
            return TMG_OK;
        if (!g->logits || !g->out || !g->x || (g->F > 0 && (!g->W1 || !g->W2)))
            return fail(TMG_ERR_INVALID_ARG, "null pointer");
        DeviceState *ds = nullptr;
        tmg_status st;
        if ((st = device_state(&ds)) != TMG_OK)
            return st;
        cudaStream_t s = static_cast<cudaStream_t>(stream);
        const StreamLock lock(s);
        return few_tokens(*g) ? moe_few(*ds, *g, s) : moe_by_groups(*ds, *g, s);
    });
}

tmg_status tmg_lora_linear(const tmg_lora_args *g, void *stream)
{
    return guarded([&]() -> tmg_status {
        if (!g)
            return fail(TMG_ERR_INVALID_ARG, "null argument struct");
        tmg_status st;
        if ((st = check_lora(g->M, g->N, g->K, g->r, g->L)) != TMG_OK)
            return st;
        if (!extents_ok(g->M, g->ldx, g->K, 1) || !extents_ok(g->N, g->ldw, g->K, 1) || !extents_ok(g->M, g->ldd, g->N, 1) ||
            !out_rows_ok(g->M, g->N, g->ldd) || (g->residual && !extents_ok(g->M, g->ld_residual, g->N, 1)))
            return fail(TMG_ERR_INVALID_ARG, "row stride of x, W, D or residual out of range");
        if (g->M == 0)
            return TMG_OK;
        if (!g->adapters || (g->K > 0 && (!g->x || !g->A)) || (g->N > 0 && (!g->D || !g->B || (g->K > 0 && !g->W))))
            return fail(TMG_ERR_INVALID_ARG, "null pointer");
        DeviceState *ds = nullptr;
        if ((st = device_state(&ds)) != TMG_OK)
            return st;
        cudaStream_t s = static_cast<cudaStream_t>(stream);
        const StreamLock lock(s);
        RankArgs k{g->x, g->A, g->adapters, g->scales, g->u, g->M, g->K, g->L, g->ldx, up(g->r, 8), static_cast<int>(g->r), false};
        const bool few = g->M <= kLoraFewRows && g->r <= kLoraFewRanks;
        const bool with = few_ranks(k) && lora_few_with(g->M, g->N, g->K, g->r, ds->num_sms);
        const int64_t ldu = k.ldu;
        if (!with && (!k.U || ldu != g->r || !aligned(k.U))) {
            k.U = workspace(kWsLayer, g->M * ldu * 2, s, &st);
            if (!k.U)
                return st;
        }
        // every copy of an operand comes before the kernel that makes u: the product runs
        // beside that one
        AdaptedArgs a{};
        Rows f{};
        if ((st = tma_rows(*ds, kWsPackA, g->x, g->ldx, g->M, g->K, g->M, s, &a.x)) != TMG_OK ||
            (g->N > 0 && (st = tma_rows(*ds, kWsPackB, g->W, g->ldw, g->N, g->K, g->N, s, &a.W)) != TMG_OK) ||
            (g->N > 0 && (st = tma_rows(*ds, kWsLayoutB, g->B, g->r, g->L * g->N, g->r, g->L * g->N, s, &a.F)) != TMG_OK) ||
            (g->K > 0 && !few_ranks(k) &&
             (st = tma_rows(*ds, kWsFactor, g->A, g->K, g->L * g->r, g->K, g->L * g->r, s, &f)) != TMG_OK) ||
            (!with && (st = run_rank(*ds, k, a.x, f, false, s)) != TMG_OK))
            return st;
        a.U = k.U;
        if (g->u && k.U != g->u) {             // the caller's own, in its layout
            k.U = g->u;
            k.ldu = g->r;
            if ((st = run_rank(*ds, k, a.x, f, false, s)) != TMG_OK)
                return st;
        }
        if (g->N == 0)
            return TMG_OK;
        a.D = g->D;
        a.adapters = g->adapters;
        a.bias = g->bias;
        a.residual = g->residual;
        a.M = g->M;
        a.N = g->N;
        a.K = g->K;
        a.r = g->r;
        a.L = g->L;
        a.ldu = ldu;
        a.ldd = g->ldd;
        a.ld_residual = g->ld_residual;
        if (few)
            return run_adapted_few(*ds, a, with ? &k : nullptr, s);
        AdaptedTiles t;
        return (st = adapted_tiles(a, ds->num_sms, &t)) != TMG_OK ? st : run_adapted(*ds, a, t, s);
    });
}

tmg_status tmg_lora_linear_backward(const tmg_lora_grad_args *g, void *stream)
{
    return guarded([&]() -> tmg_status {
        if (!g)
            return fail(TMG_ERR_INVALID_ARG, "null argument struct");
        tmg_status st;
        if ((st = check_lora(g->M, g->N, g->K, g->r, g->L)) != TMG_OK)
            return st;
        if (!extents_ok(g->M, g->ldd, g->N, 1) || !extents_ok(g->M, g->ldx, g->K, 1) || !extents_ok(g->N, g->ldw, g->K, 1))
            return fail(TMG_ERR_INVALID_ARG, "row stride of dD, x or W out of range");
        const bool in = g->M > 0;
        if ((in && !g->adapters) || (in && g->N > 0 && !g->dD))
            return fail(TMG_ERR_INVALID_ARG, "null pointer (adapters or dD)");
        if (in && g->N > 0 && ((g->dx && g->K > 0 && (!g->W || !g->A || !g->B)) || (g->dA && g->K > 0 && (!g->x || !g->B)) ||
                               (g->dB && !g->u)))
            return fail(TMG_ERR_INVALID_ARG, "null pointer: dx needs W, A and B, dA needs x and B, dB needs u");
        DeviceState *ds = nullptr;
        if ((st = device_state(&ds)) != TMG_OK)
            return st;
        cudaStream_t s = static_cast<cudaStream_t>(stream);
        const StreamLock lock(s);
        const bool want_a = g->dA && g->K > 0, want_b = g->dB && g->N > 0;
        if (!in || g->N == 0) {                // no row, or no gradient of any
            if (want_a && (st = launched(cudaMemsetAsync(g->dA, 0, static_cast<size_t>(g->L) * g->r * g->K * 2, s),
                                         "cudaMemsetAsync(dA)")) != TMG_OK)
                return st;
            if (want_b && (st = launched(cudaMemsetAsync(g->dB, 0, static_cast<size_t>(g->L) * g->r * g->N * 2, s),
                                         "cudaMemsetAsync(dB)")) != TMG_OK)
                return st;
            return g->dx && in && g->K > 0 ? launched(cudaMemsetAsync(g->dx, 0, static_cast<size_t>(g->M) * g->K * 2, s),
                                                      "cudaMemsetAsync(dx)")
                                           : TMG_OK;
        }
        const bool want_x = g->dx && g->K > 0;
        const int64_t ldu = up(g->r, 8);
        Pieces p;
        const size_t du_at = p.take(g->M * ldu * 2), rows = p.take(g->M * 4), offsets = p.take((g->L + 1) * 4);
        char *ws = static_cast<char *>(workspace(kWsLayer, p.bytes, s, &st));
        if (!ws)
            return st;
        const Rows dU{ws + du_at, ldu};
        // copies of operands first: dx's kernel runs beside the one that makes dU, and
        // that one beside the plan's
        AdaptedArgs a{};
        LoraGradArgs grads;
        std::memset(&grads, 0, sizeof grads);
        Rows x{}, u{}, f{};
        if ((st = tma_rows(*ds, kWsPackA, g->dD, g->ldd, g->M, g->N, g->M, s, &a.x)) != TMG_OK ||
            (want_x && ((st = tma_rows(*ds, kWsPackB, g->W, g->ldw, g->N, g->K, g->N, s, &a.W)) != TMG_OK ||
                        (st = tma_rows(*ds, kWsLayoutB, g->A, g->K, g->L * g->r, g->K, g->L * g->r, s, &a.F)) != TMG_OK)) ||
            ((want_x || want_a) && (st = tma_rows(*ds, kWsFactor, g->B, g->r, g->L * g->N, g->r, g->L * g->N, s, &f)) != TMG_OK) ||
            (want_a && ((st = tma_rows(*ds, kWsGather, g->x, g->ldx, g->M, g->K, g->M, s, &x)) != TMG_OK ||
                        (st = grad_side(grads.side[grads.sides++], x, g->K, dU, g->M, g->dA, false)) != TMG_OK)) ||
            (want_b && ((st = tma_rows(*ds, kWsLayoutA, g->u, g->r, g->M, g->r, g->M, s, &u)) != TMG_OK ||
                        (st = grad_side(grads.side[grads.sides++], a.x, g->N, u, g->M, g->dB, true)) != TMG_OK)))
            return st;
        if (grads.sides) {
            grads.offsets = reinterpret_cast<int32_t *>(ws + offsets);
            grads.rows = reinterpret_cast<int32_t *>(ws + rows);
            grads.M = static_cast<int>(g->M);
            grads.L = static_cast<int>(g->L);
            grads.r = static_cast<int>(g->r);
            if ((st = launched(launch_lora_plan(g->adapters, grads.M, grads.L, reinterpret_cast<int32_t *>(ws + offsets),
                                                reinterpret_cast<int32_t *>(ws + rows), s),
                               "row plan launch")) != TMG_OK)
                return st;
        }
        if ((want_x || want_a) &&
            (st = run_rank(*ds, RankArgs{g->dD, g->B, g->adapters, g->scales, ws + du_at, g->M, g->N, g->L, g->ldd, ldu,
                                         static_cast<int>(g->r), true},
                           a.x, f, grads.sides > 0, s)) != TMG_OK)
            return st;
        // Factors first where their CTAs and dx's fit the GPU at once: dx's product then runs
        // beside them and waits for them and dU (700 rows of 2 adapters of rank 64, 4096 x
        // 2048, 35.0 -> 29.9 us; 700 x 4096 x 4096, where they do not fit, 43.4 and 47.6).
        AdaptedTiles t{};
        if (want_x) {
            a.U = dU.p;
            a.D = g->dx;
            a.adapters = g->adapters;
            a.M = g->M;
            a.N = a.ldd = g->K;
            a.K = g->N;
            a.r = g->r;
            a.L = g->L;
            a.ldu = ldu;
            a.across = true;
            if ((st = adapted_tiles(a, ds->num_sms, &t)) != TMG_OK)
                return st;
        }
        const bool first = grads.sides && !t.split && lora_grad_ctas(grads, ds->num_sms) + t.ctas <= ds->num_sms;
        if ((first && (st = run_grad(*ds, grads, s)) != TMG_OK) || (want_x && (st = run_adapted(*ds, a, t, s)) != TMG_OK))
            return st;
        return grads.sides && !first ? run_grad(*ds, grads, s) : TMG_OK;
    });
}

}  // extern "C"
