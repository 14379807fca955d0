// lora.h — arguments of the kernels of dense projections with low-rank adapters.
#pragma once

#include "few.cuh"

namespace tmg {

// U[m][j] = bf16(scales[a] sum_c X[m][c] F[a][j][c]) with a = adapters[m], or, `across`,
// of F[a][c][j]; zeros where a is not one of 0 .. L - 1.  F is contiguous, (L, r, C) or
// (L, C, r).
struct RankArgs {
    const void *X, *F;
    const int32_t *adapters;
    const float *scales;       // (L) or null (ones)
    void *U;                   // bf16 (M, r), row stride ldu
    int64_t M, C, L, ldx, ldu;
    int r;
    bool across;
};
// For a few rows: not across, C a multiple of 8, X's and F's rows 16-byte aligned.
cudaError_t launch_lora_few_rank(const RankArgs &a, int num_sms, cudaStream_t s);

// The same on the tensor cores.
struct LoraRankArgs {
    CUtensorMap tmX;           // (M, C): 128 rows of 64
    CUtensorMap tmF;           // (L, r, C): r rounded up to 16 rows of 64; maj: (L, C, r), 64 x 64
    const int32_t *adapters;
    const float *scales;
    void *U;
    int64_t ldu;
    int M, C, L, r;
    int beside;                // the kernel before leaves X, F and the adapters alone: no wait for it
    // set by the launch
    int cluster, chunk, block_bytes, stages, stage_bytes, ring_bytes, tmem_cols;
};
cudaError_t launch_lora_rank_tc(LoraRankArgs a, bool maj, int num_sms, const ErrCtx &err, cudaStream_t s);

// D[m] = x[m] . W^T + U[m] . F[adapters[m]]^T + bias + residual[m] for at most
// kLoraFewRows rows and kLoraFewRanks ranks (the factors of 32 columns of every warp,
// U and the results must fit shared memory beside the ring).
// With A given, U is made by the same kernel, where lora_few_with() holds.
constexpr int kLoraFewRows = 64, kLoraFewRanks = 128, kLoraFewWith = 32;
struct LoraFewArgs {
    CUtensorMap tmW;           // (N, K): 128 rows of 64
    CUtensorMap tmX;           // (M, K): shape.tp rows of 64
    const void *F;             // (L, N) rows of ldf, 16-byte aligned
    void *U;                   // rows of ldu, 16-byte aligned; with A: (M, r), written, or null
    const void *X, *A;         // with A: rows of ldx and (L, r, K), 16-byte aligned, K a multiple of 8
    const float *scales;       // or null
    void *D;
    const int32_t *adapters;
    const float *bias;
    const void *residual;
    int64_t ldu, ldx, ldf, ldd, ld_residual;
    int M, N, K, L, r;
    FewShape shape;            // tp; the rest is set by the launch
    int room_bytes;            // set by the launch
};
bool lora_few_with(int64_t M, int64_t N, int64_t K, int64_t r, int num_sms);
cudaError_t launch_lora_few(LoraFewArgs a, int num_sms, const ErrCtx &err, cudaStream_t s);

// D[m] = x[m] . W^T + U[m] . F[adapters[m]]^T + bias + residual[m] on CTA pairs, or with
// W (K, N) and F (L, r, N) given along their rows (`maj`).
struct LoraPairArgs {
    CUtensorMap tmX, tmU;      // (M, K), (M, r): boxes of 128 rows of 64
    CUtensorMap tmW;           // (N, K): bn / 2 rows of 64; maj: (K, N), 64 x 64
    CUtensorMap tmF;           // (L, N, r): bn / 2 rows of 64; maj: (L, r, N), 64 x 64
    void *D;
    const int32_t *adapters;
    const float *bias;         // or null
    const void *residual;      // or null
    int64_t ldd, ld_residual;
    int M, N, K, L, r;
    int vec_ok;                // rows of D are 16-byte aligned
    int group_m;               // row tiles per band
    int cut_tiles, cut_pieces; // swap_time's
    float *partials;           // of cut tiles: sw_partial_floats(bn) per pair
    uint32_t *counters;        // 16 per cut tile
    uint32_t *feed;            // the tile counter
};
// The same in tiles of 128 x 128 over clusters (W and F K-major: boxes of 128 rows).
cudaError_t launch_lora_split(const LoraPairArgs &a, bool maj, int cluster, const ErrCtx &err, cudaStream_t s);
cudaError_t launch_lora_pair(const LoraPairArgs &a, int bn, bool maj, int pairs, const ErrCtx &err, cudaStream_t s);

// The rows sorted by adapter: adapter l's are rows[offsets[l]] .. rows[offsets[l + 1] - 1],
// in order.  Reads only the adapters and lets its successor start at once.
cudaError_t launch_lora_plan(const int32_t *adapters, int M, int L, int32_t *offsets, int32_t *rows, cudaStream_t s);

// G[l] = sum over the rows m of adapter l of Z[m]^T Y[m], (L, r, C), or, `across`, its
// transpose (L, C, r); contiguous, zeros for an adapter without rows.
struct LoraGradSide {
    CUtensorMap tmY[3];        // (M, C): boxes of 64 columns by 64, 16 and one rows
    const void *Z;             // (M, r), 16-byte rows of ldz
    int64_t ldz;
    void *G;
    int C, across;
};
struct LoraGradArgs {
    LoraGradSide side[2];
    int sides;                         // 1 or 2
    const int32_t *offsets, *rows;     // launch_lora_plan's
    int M, L, r;
    float *partials;                   // lora_grad_partial_bytes()
    uint32_t *counters;                // lora_grad_counters(), zero between launches
    int runs, stages, stage_bytes, tmem_cols;     // set by the launch
};
int64_t lora_grad_ctas(const LoraGradArgs &a, int num_sms);
size_t lora_grad_partial_bytes(const LoraGradArgs &a, int num_sms);
size_t lora_grad_counters(const LoraGradArgs &a, int num_sms);
cudaError_t launch_lora_grad(LoraGradArgs a, int num_sms, const ErrCtx &err, cudaStream_t s);

}  // namespace tmg
