// moe_few.cu — a whole expert layer for a few tokens, in two kernels: the choice of
// the experts with the gate and up products and SwiGLU, then the down products with the
// weighted sum and the residual.
//
// With few tokens the layer is the reading of the chosen experts' weights.  Both
// kernels take 128 weight rows as the MMA's M and all T tokens (padded to tp, a
// multiple of 16) as its N, for every expert that any token chose: nothing is sorted,
// gathered or grouped, and a tile needs no more than its expert's number.
//
// Choice.  Up to 16 tokens every CTA chooses all tokens' experts from the logits by
// itself (a warp per token, route.cuh), which takes it less time than a kernel of its
// own would; for more there is one.
//
// First kernel.  A tile is 64 gate rows and their 64 up rows of one chosen expert.
// hidden[i][t] = bf16(w[t, e] silu(g) u) for the i-th chosen expert e, zeros for tokens
// that did not choose it: the weight is folded in, so that
//
// the second kernel's sum over experts is one long contraction, out[t] = sum over (i, f)
// of W2[e_i][:, f] hidden[i][t][f]: a tile of 128 columns of the layer's output
// accumulates all chosen experts one after another.  A zero times a weight that is
// infinite or NaN would be NaN in a token that did not choose that expert: where a sum
// comes out as NaN, it is formed again from the token's own experts alone, by a warp for
// eight columns (few_again()).
//
// Where tiles are few, a cluster of CTAs splits a tile's contraction, and the partial sums
// meet in shared memory as in split_kernel.cuh.  Two CTAs fit an SM.  The second kernel starts
// while the first one runs: it finds the experts as that one does and fills its ring with
// W2's first blocks, and only the hidden rows wait for the first kernel's end.  The
// first one lets it start only after its own wait for the kernel before: so logits (or
// choices) and weights are complete by then.
//
// Bound by HBM: 13 tokens, 4 of 32 experts, 4096 x 2048, 20 to 22 in use, 1.07 GB, 168 to
// 172 us (6.3 TB/s); one token's 8 of 64 experts, 2048 x 1024, 101 MB, 25.8 us, of them 2
// for the choice, 13 for the first kernel's stream (6.1 TB/s, W2's first blocks in it), 1
// until the second one learns of its end, 6 for the rest of W2 and 1 for the sums.
#include <atomic>

#include "act.cuh"
#include "few.cuh"
#include "moe_few.h"
#include "route.cuh"
#include "staging.cuh"

namespace tmg {
namespace {

constexpr int kFwThreads = 256;

struct FewSmem : FewRing {
    int chosen;                              // experts with a token
    float weights[kFewTokens * kFewChoices];
    int32_t experts[kFewTokens * kFewChoices];
    int32_t counts[kFewExperts];
    int32_t list[kFewExperts];               // the chosen experts, smallest first
    uint32_t tokens[kFewExperts][2];         // which tokens chose them

    __device__ __forceinline__ bool chose(int i, int t) const { return tokens[i][t >> 5] >> (t & 31) & 1u; }
    float weight[kFewTokens];                // first kernel: of its expert
};

// Before few_choose().
__device__ __forceinline__ void few_clear(FewSmem &sm)
{
    for (int i = threadIdx.x; i < kFewExperts; i += kFwThreads) {
        sm.counts[i] = 0;
        sm.tokens[i][0] = sm.tokens[i][1] = 0;
    }
    __syncthreads();
}

__device__ __forceinline__ RouteArgs few_route(const MoeFewArgs &p, float *weights, int32_t *experts)
{
    RouteArgs r{};
    r.logits = p.logits;
    r.T = p.T;
    r.ld = p.ld_logits;
    r.E = p.E;
    r.k = p.k;
    r.normalize = p.normalize;
    r.weights = weights;
    r.experts = experts;
    return r;
}

// The choices of many tokens, a warp per token.
constexpr int kFwChoosers = 8;
template <int C, bool BF16>
__global__ void __launch_bounds__(32 * kFwChoosers) moe_few_choose_kernel(MoeFewArgs p)
{
    __shared__ int32_t counts[kFewExperts];      // no one reads them here
    grid_wait();
    grid_release();
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kFwChoosers;
    choose<C, BF16>(few_route(p, p.weights, p.chosen), t0, min(static_cast<int64_t>(p.T), t0 + kFwChoosers), counts, nullptr);
}

// All threads: choose the tokens' experts (C = 0: read the choices).
template <int C, bool BF16>
__device__ __forceinline__ void few_choose(const MoeFewArgs &p, FewSmem &sm)
{
    if constexpr (C == 0) {
        for (int i = threadIdx.x; i < p.T * p.k; i += kFwThreads) {
            const int e = __ldcg(p.chosen + i);
            sm.experts[i] = e;
            sm.weights[i] = __ldcg(p.weights + i);
            if (e >= 0)
                atomicAdd(&sm.counts[e], 1);
        }
    } else {
        choose<C, BF16, true>(few_route(p, sm.weights, sm.experts), 0, p.T, sm.counts, nullptr);
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        int n = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + threadIdx.x;
            const bool on = e < p.E && sm.counts[e] > 0;
            const uint32_t all = __ballot_sync(0xffffffffu, on);
            if (on) {
                const int at = n + __popc(all & ((1u << threadIdx.x) - 1));
                sm.list[at] = e;
                sm.counts[e] = at;               // its place
            }
            n += __popc(all);
        }
        if (threadIdx.x == 0)
            sm.chosen = n;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.T * p.k; i += kFwThreads) {
        const int e = sm.experts[i], t = i / p.k;
        if (e >= 0)
            atomicOr(&sm.tokens[sm.counts[e]][t >> 5], 1u << (t & 31));
    }
    __syncthreads();
}

// The four epilogue warps meet; whether any of their threads says so.
__device__ __forceinline__ bool few_epilogue_any(bool mine)
{
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "barrier.cta.red.or.pred p, 1, 128, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(any)
        : "r"(mine ? 1u : 0u)
        : "memory");
    return any != 0;
}

// The tile of the i-th chosen expert's columns f0 ..: sum of the cluster's partial
// sums, SwiGLU, weight; eight columns of a token per thread, items x, x + step, ...
__device__ __forceinline__ void few_hidden(const MoeFewArgs &p, const FewSmem &sm, uint32_t sums, uint32_t S, int i, int f0, int x,
                                           int items, int step, const ErrCtx &err)
{
    const int64_t limit = static_cast<int64_t>(min(p.E, p.T * p.k)) * p.shape.tp * p.F;
    for (; x < items; x += step) {
        const int t = x / 8, c = x % 8 * 8, f = f0 + c, n = min(8, p.F - f);
        if (n <= 0)
            continue;
        float g[8] = {}, u[8];
        if (t < p.T && sm.chose(i, t)) {
            const float w = sm.weight[t];
            few_sum(sums, t, c, S, g);
            few_sum(sums, t, 64 + c, S, u);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                g[j] = w * (silu_f(g[j]) * u[j]);
        }
        store_piece(static_cast<__nv_bfloat16 *>(p.hidden), (static_cast<int64_t>(i) * p.shape.tp + t) * p.F + f,
                    make_uint4(pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3]), pack_bf16x2(g[4], g[5]), pack_bf16x2(g[6], g[7])),
                    n, limit, err);
    }
}

template <int C, bool BF16>
__global__ void __launch_bounds__(kFwThreads, 2) moe_few_up_kernel(const __grid_constant__ MoeFewArgs p, ErrCtx err)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ FewSmem sm;
    __shared__ uint64_t tfull[2], tempty[2];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t *ring = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    float *staged = reinterpret_cast<float *>(ring + p.shape.ring_bytes);        // a tile's sums [token][128]
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    volatile int *abort_flag = &sm.abort;
    if (threadIdx.x == 0)
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], 4);
        }
    few_setup(p.shape, sm, &p.tmW1, &p.tmX);
    few_clear(sm);
    grid_wait();
    grid_release();
    few_choose<C, BF16>(p, sm);
    tc_fence_after();
    const uint32_t tmem = sm.tmem_slot;
    const uint32_t rank = cluster_ctarank(), S = few_cluster_size();
    const int f_tiles = ceil_div(p.F, 64), num_kb = ceil_div(p.H, 64), tiles = sm.chosen * f_tiles;
    const int first = blockIdx.x / S, step = gridDim.x / S;        // this cluster's tiles: one at most where it is not one CTA
    const int kb0 = static_cast<int>(static_cast<int64_t>(num_kb) * rank / S);
    const int kb1 = static_cast<int>(static_cast<int64_t>(num_kb) * (rank + 1) / S);

    if (warp == 0 || warp == 2) {
        // ------------------ TMA producers: the weights (warp 0), the rows (warp 2)
        int stage = 0, issued = 0;
        uint32_t phase = 0;
        bool ok = true;
        const uint32_t tx = kFwWeights + static_cast<uint32_t>(p.shape.tp) * 128u;
        for (int tile = first; ok && tile < tiles; tile += step) {
            const int e = sm.list[tile / f_tiles], f0 = tile % f_tiles * 64;
            for (int kb = kb0; kb < kb1; ++kb, ++issued) {
                if (!mbar_wait_warp(&sm.empty[stage], phase ^ 1u, err, abort_flag, kSiteProducerEmpty)) {
                    ok = false;
                    break;
                }
                uint8_t *at = ring + stage * p.shape.stage_bytes;
                if (warp == 0) {
                    mbar_arrive_expect_tx_w(&sm.full[stage], tx);
                    tma_load_3d_one(at, &p.tmW1, &sm.full[stage], kb * 64, f0, e);
                    tma_load_3d_one(at + kFwWeights / 2, &p.tmW1, &sm.full[stage], kb * 64, p.F + f0, e);
                } else {
                    tma_load_2d_w(at + kFwWeights, &p.tmX, &sm.full[stage], kb * 64, 0);
                }
                if (++stage == p.shape.stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        for (int i = 0; i < p.shape.stages && i < issued; ++i) {          // every stage is released
            const int s = stage - 1 - i;
            mbar_wait(&sm.empty[s < 0 ? s + p.shape.stages : s], s < 0 ? phase ^ 1u : phase, err, abort_flag, kSiteDrain);
        }
        if (lane == 0)
            sm.issued[warp / 2] = issued;
    } else if (warp == 1) {
        // -------------------------------------------- MMA issuer
        const uint32_t idesc = idesc_bf16_f32(128, p.shape.tp);
        int stage = 0, local = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int tile = first; ok && tile < tiles; tile += step) {
            const int acc = local & 1;
            const uint32_t acc_phase = (local >> 1) & 1;
            ++local;
            if (!mbar_wait_warp(&tempty[acc], acc_phase ^ 1u, err, abort_flag, kSiteMmaTmemEmpty))
                break;
            tc_fence_after();
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!mbar_wait_warp(&sm.full[stage], phase, err, abort_flag, kSiteMmaFull)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t w_s = smem_u32(ring + stage * p.shape.stage_bytes);
                const uint64_t wdesc = sdesc_kmajor_sw128(w_s), rdesc = sdesc_kmajor_sw128(w_s + kFwWeights);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_bf16_w(tmem + acc * 64, wdesc + k * 2, rdesc + k * 2, idesc, (kb != kb0) || (k != 0));
                mma_commit_w(&sm.empty[stage]);
                if (++stage == p.shape.stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok)
                break;
            mma_commit_w(&tfull[acc]);
        }
        if (*abort_flag)
            settle(sm.empty, p.shape.stages, stage, phase, 1, err.word, err.budget_ns);
    } else if (warp >= 4) {
        // ---------------------------------------------------- epilogue
        const int q = warp & 3, id = threadIdx.x - 128;
        int local = 0;
        for (int tile = first; tile < tiles; tile += step) {
            const int acc = local & 1, e = sm.list[tile / f_tiles];
            const uint32_t acc_phase = (local >> 1) & 1;
            ++local;
            for (int j = id; j < p.T * p.k; j += 128)        // the last tile's reads are done
                if (sm.experts[j] == e)
                    sm.weight[j / p.k] = sm.weights[j];
            const bool there = mbar_wait_warp(&tfull[acc], acc_phase, err, abort_flag, kSiteEpiTmemFull);
            tc_fence_after();
            if (there)
                for (int c = 0; c < p.shape.tp; c += 16) {
                    uint32_t r[16];
                    tmem_ld16(tmem + (static_cast<uint32_t>(q * 32) << 16) + acc * 64 + c, r);
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        staged[(c + j) * 128 + q * 32 + lane] = __uint_as_float(r[j]);
                }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&tempty[acc]);
            if (S > 1)
                break;
            if (few_epilogue_any(!there))                    // a wait ran out: all leave together
                break;
            few_hidden(p, sm, smem_u32(staged), 1, tile / f_tiles, tile % f_tiles * 64, id, p.shape.tp * 8, 128, err);
            few_epilogue_any(false);                         // the staged tile and the weights are free
        }
    }
    __syncwarp();
    if (S > 1) {                                             // the cluster's partial sums meet
        cluster_sync();
        const int items = p.shape.tp * 8;
        if (first < tiles && !*abort_flag)
            few_hidden(p, sm, smem_u32(staged), S, first / f_tiles, first % f_tiles * 64, items * rank / S + threadIdx.x,
                       items * (rank + 1) / S, kFwThreads, err);
        cluster_sync();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0 && *abort_flag) {
        const int n = few_announce(p.shape, sm);
        settle(sm.full, p.shape.stages, n % p.shape.stages, n / p.shape.stages & 1, n, err.word, err.budget_ns);
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, p.shape.tmem_cols);
    }
}

// Columns col .. col + n - 1 of token t's residual, zeros without one; past L1, since the
// first ones are read before the kernel's own wait.
__device__ __forceinline__ void few_residual(const MoeFewArgs &p, int t, int col, int n, bool on, float (&f)[8])
{
    const __nv_bfloat16 *res = static_cast<const __nv_bfloat16 *>(p.residual);
    const __nv_bfloat16 *r = res + t * p.ld_residual + col;
    const bool wide = res && on && n == 8 && (reinterpret_cast<uintptr_t>(r) & 15u) == 0;
    const uint4 v = wide ? __ldcg(reinterpret_cast<const uint4 *>(r)) : make_uint4(0, 0, 0, 0);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(w[j] << 16);
        f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
    if (res && on && !wide)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            f[j] = j < n ? __uint_as_float(static_cast<uint32_t>(__ldcg(reinterpret_cast<const unsigned short *>(r + j))) << 16) : 0.f;
}

// Eight columns of a token's result: sum + residual, rounded.
__device__ __forceinline__ void few_store(const MoeFewArgs &p, int t, int col, int n, const float (&z)[8], const float (&add)[8],
                                          const ErrCtx &err)
{
    store_piece(static_cast<__nv_bfloat16 *>(p.out), t * p.ld_out + col,
                make_uint4(pack_bf16x2(z[0] + add[0], z[1] + add[1]), pack_bf16x2(z[2] + add[2], z[3] + add[3]),
                           pack_bf16x2(z[4] + add[4], z[5] + add[5]), pack_bf16x2(z[6] + add[6], z[7] + add[7])),
                n, (p.T - 1) * p.ld_out + p.H, err);
}

// The results of this CTA with a NaN among their eight columns, a warp for each.  Where the
// token's own hidden values hold a NaN, that is the sum, whatever the weights hold;
// else its NaN columns are formed again from its own experts, 256 elements of all
// eight columns a step.  Out of line: no call reaches it unless a sum is NaN.  8 of 64
// experts, 2048 x 1024, a NaN in one token's x: one token 23 -> 27 us, 61 tokens 145 -> 155
// (a thread for eight columns, 1126 and 2523); all weights of eight experts that one
// of 61 tokens chose infinite, so that every other token's row is formed again, 2.1 ms.
static __device__ __noinline__ void few_again(const MoeFewArgs &p, const FewSmem &sm, const uint8_t *again, uint32_t part, uint32_t S,
                                              int n0, int first, int last, const ErrCtx &err)
{
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const __nv_bfloat16 *hidden = static_cast<const __nv_bfloat16 *>(p.hidden), *W2 = static_cast<const __nv_bfloat16 *>(p.W2);
    int token = -1;
    bool own = false;                        // the token's hidden values hold a NaN
    for (int x = first + warp; x < last; x += kFwThreads / 32) {
        if (!again[x - first])
            continue;
        const int t = x / 16, c = x % 16 * 8, col = n0 + c, n = min(8, p.H - col);
        if (t != token) {
            token = t;
            bool nan = false;
            for (int i = 0; i < sm.chosen; ++i)
                if (sm.chose(i, t)) {
                    const __nv_bfloat16 *h = hidden + (static_cast<int64_t>(i) * p.shape.tp + t) * p.F;
#pragma unroll 4
                    for (int f = lane * 8; f < p.F; f += 256) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(h + f);
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            nan |= (w[j] & 0x7fffu) > 0x7f80u || (w[j] & 0x7fff0000u) > 0x7f800000u;
                    }
                }
            own = __any_sync(0xffffffffu, nan);
        }
        float z[8], add[8];
        few_sum(part, t, c, S, z);
        few_residual(p, t, col, n, true, add);
        if (!own) {
            float sum[8] = {};
            for (int i = 0; i < sm.chosen; ++i)
                if (sm.chose(i, t)) {
                    const __nv_bfloat16 *w = W2 + (static_cast<int64_t>(sm.list[i]) * p.H + col) * p.F;
                    const __nv_bfloat16 *h = hidden + (static_cast<int64_t>(i) * p.shape.tp + t) * p.F;
                    for (int f = lane * 8; f < p.F; f += 256) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(h + f);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (j < n && z[j] != z[j])
                                sum[j] = dot8(*reinterpret_cast<const uint4 *>(w + j * static_cast<int64_t>(p.F) + f), v, sum[j]);
                    }
                }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
#pragma unroll
                for (int o = 16; o; o >>= 1)
                    sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], o);
                z[j] = z[j] != z[j] ? sum[j] : z[j];
            }
        }
        if (lane == 0)
            few_store(p, t, col, n, z, add, err);
    }
}

template <int C, bool BF16>
__global__ void __launch_bounds__(kFwThreads, 2) moe_few_down_kernel(const __grid_constant__ MoeFewArgs p, ErrCtx err)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ FewSmem sm;
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t *ring = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    const uint32_t rank = cluster_ctarank(), S = few_cluster_size();
    const int n0 = blockIdx.x / S * 128;
    few_setup(p.shape, sm, &p.tmW2, &p.tmHidden);
    few_clear(sm);
    grid_release();
    few_choose<C, BF16>(p, sm);
    tc_fence_after();
    const int per = ceil_div(p.F, 64), num_kb = sm.chosen * per;
    const int kb0 = static_cast<int>(static_cast<int64_t>(num_kb) * rank / S);
    const int kb1 = static_cast<int>(static_cast<int64_t>(num_kb) * (rank + 1) / S);
    // this CTA's share of the results, eight columns of a token at a time, the free
    // warps first; the residual is read ahead
    const int items = p.T * 16, first = items * rank / S, last = items * (rank + 1) / S;
    const int item0 = first + (threadIdx.x + kFwThreads / 2) % kFwThreads;
    auto read = [&](int x, float (&f)[8]) {
        const int col = n0 + x % 16 * 8;
        few_residual(p, x / 16, col, min(8, p.H - col), x < last, f);
    };
    float add[8];
    few_product(
        p.shape, sm, ring, kb0, kb1,
        [&](uint8_t *dst, uint64_t *bar, int kb) { tma_load_3d_one(dst, &p.tmW2, bar, kb % per * 64, n0, sm.list[kb / per]); },
        [&](uint8_t *dst, uint64_t *bar, int kb) { tma_load_3d_one(dst, &p.tmHidden, bar, kb % per * 64, 0, kb / per); },
        [] { grid_wait(); }, [&] { read(item0, add); }, err);
    if (threadIdx.x < kFwThreads / 2)
        read(item0, add);
    grid_wait();                     // every warp: the first kernel's hidden rows
    const uint32_t part = smem_u32(ring);
    uint8_t *again = reinterpret_cast<uint8_t *>(sm.counts);       // of each result: it has a NaN
    static_assert(kFewTokens * 16 <= sizeof(sm.counts), "a byte per result of a CTA");
    bool any = false;
    for (int x = item0; x < last; x += kFwThreads) {
        const int t = x / 16, c = x % 16 * 8, col = n0 + c, n = min(8, p.H - col);
        bool nan = false;
        if (n > 0) {
            if (x != item0)
                read(x, add);
            float z[8];
            few_sum(part, t, c, S, z);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                nan |= j < n && z[j] != z[j];
            if (!nan)
                few_store(p, t, col, n, z, add, err);
        }
        again[x - first] = nan;
        any |= nan;
    }
    if (__syncthreads_or(any))
        few_again(p, sm, again, part, S, n0, first, last, err);
    __syncwarp();
    cluster_sync();                  // no CTA leaves while its partial sums may be read
}

// The clusters of four CTAs that run at once with an SM for each: a cluster stays within
// a part of the chip whose SMs need not be a multiple of four (36 on 152 SMs).
int quads_at_once()
{
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return 0;
    int n = known[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        const int smem = 1024 + 2 * kFwRing - 16384;
        auto kern = moe_few_down_kernel<0, false>;
        cudaLaunchAttribute cluster = {};
        cluster.id = cudaLaunchAttributeClusterDimension;
        cluster.val.clusterDim.x = 4;
        cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(4);
        cfg.blockDim = dim3(kFwThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.attrs = &cluster;
        cfg.numAttrs = 1;
        if (ensure_smem_attr(reinterpret_cast<const void *>(kern), smem) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
            (void)cudaGetLastError();                    // not an error of the next launch
            return 0;
        }
        known[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

template <int C, bool BF16>
cudaError_t launch_few_as(MoeFewArgs a, int num_sms, const ErrCtx &err, cudaStream_t s)
{
    // Half an SM's shared memory each, so that the second kernel starts beside the first;
    // with many tokens, and so much to read, the first one takes all of an SM's (61 tokens
    // of 64 experts, 2048 x 1024: 143 us against 152).
    MoeFewArgs b = a;
    few_ring(a.shape, C == 0 ? 2 * kFwRing - a.shape.tp * 512 : kFwRing);
    // The second kernel: two CTAs per SM in clusters of up to eight, with these exceptions.
    // Clusters of four where those take three quarters of the SMs at one CTA each: with all
    // of an SM's shared memory if they all fit at once so (4 of 32 experts, width 1024, 35
    // tiles, 13 tokens 122 -> 118 us, 61 tokens 169 -> 147; width 2048, 32 tiles, 13 tokens 205
    // and 204; 25 tiles 90 and 94), else with half of it (38 tiles, where 36 clusters fit:
    // 157 us with all of it, 144 in clusters of eight, 127 so).  Pairs with an SM for each
    // CTA where clusters of four do not all fit at two per SM (4 of 16 experts, 75 tiles,
    // 13 tokens 170 -> 152, one token's 2 of 8 experts 34 -> 30; 68 tiles, where they fit, 28.0
    // and 29.2 in pairs).
    const int64_t downs = (a.H + 127) / 128;
    const bool four = 4 * downs <= num_sms && 16 * downs >= 3 * num_sms;
    const bool pairs = 2 * downs <= num_sms && 8 * downs >= 3 * num_sms;
    const int quads = four || pairs ? quads_at_once() : 0;
    const bool two = pairs && downs > 2 * quads, deep = two || (four && downs <= quads);
    const int s_down = four ? 4 : two ? 2 : few_cluster(downs, static_cast<int64_t>(a.k) * ((a.F + 63) / 64), 2 * num_sms);
    few_ring(b.shape, deep ? 2 * kFwRing - 16384 : kFwRing);
    const int smem = 1024 + b.shape.ring_bytes, smem_up = 1024 + a.shape.ring_bytes + a.shape.tp * 512;
    auto up = moe_few_up_kernel<C, BF16>;
    auto down = moe_few_down_kernel<C, BF16>;
    cudaError_t e;
    if ((e = ensure_smem_attr(reinterpret_cast<const void *>(up), smem_up)) != cudaSuccess ||
        (e = ensure_smem_attr(reinterpret_cast<const void *>(down), smem)) != cudaSuccess)
        return e;
    // The first kernel: a CTA per SM over all tiles, or a cluster for each where there
    // are few (one token's 2 of 8 experts, 4096 -> 2 x 2048, 64 tiles: 27.0 us
    // against 30.1).
    const int experts = a.T * a.k < a.E ? a.T * a.k : a.E;
    const int64_t ups = static_cast<int64_t>(experts) * ((a.F + 63) / 64);
    const int s_up = few_cluster(ups, (a.H + 63) / 64, num_sms);
    if ((e = launch_overlapped(up, dim3(static_cast<unsigned>(s_up > 1 ? ups * s_up : num_sms)), kFwThreads, smem_up, s_up, s, a,
                               err)) != cudaSuccess)
        return e;
    return launch_overlapped(down, dim3(static_cast<unsigned>(downs * s_down)), kFwThreads, smem, s_down, s, b, err);
}

template <int C, bool BF16>
cudaError_t launch_few_choice(const MoeFewArgs &a, int num_sms, const ErrCtx &err, cudaStream_t s)
{
    if (a.T <= kFewOwnChoice)
        return launch_few_as<C, BF16>(a, num_sms, err, s);
    const cudaError_t e = launch_overlapped(moe_few_choose_kernel<C, BF16>, dim3((a.T + kFwChoosers - 1) / kFwChoosers),
                                            32 * kFwChoosers, 0, 1, s, a);
    return e != cudaSuccess ? e : launch_few_as<0, false>(a, num_sms, err, s);
}

template <int C>
cudaError_t launch_few_of(const MoeFewArgs &a, int num_sms, const ErrCtx &err, cudaStream_t s)
{
    return a.bf16 ? launch_few_choice<C, true>(a, num_sms, err, s) : launch_few_choice<C, false>(a, num_sms, err, s);
}

}  // namespace

cudaError_t launch_moe_few(MoeFewArgs a, int num_sms, const ErrCtx &err, cudaStream_t s)
{
    a.shape.tmem_cols = 128;
    return a.E <= 64    ? launch_few_of<2>(a, num_sms, err, s)
           : a.E <= 128 ? launch_few_of<4>(a, num_sms, err, s)
                        : launch_few_of<8>(a, num_sms, err, s);
}

}  // namespace tmg
