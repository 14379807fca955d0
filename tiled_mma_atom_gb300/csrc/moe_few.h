// moe_few.h — arguments of the two kernels that run a whole expert layer for a few
// tokens (moe_few.cu).
#pragma once

#include "few.cuh"

namespace tmg {

// Tokens of the two kernels, and those whose experts every CTA chooses by itself.
constexpr int kFewTokens = 64, kFewOwnChoice = 16, kFewExperts = 256, kFewChoices = 16;

struct MoeFewArgs {
    CUtensorMap tmW1;          // (E, 2 F, H): 64 rows of 64
    CUtensorMap tmX;           // (T, H): tp rows of 64
    CUtensorMap tmW2;          // (E, H, F): 128 rows of 64
    CUtensorMap tmHidden;      // (experts, tp, F): tp rows of 64
    const void *logits, *W2, *residual;
    float *weights;            // with more than kFewOwnChoice tokens: the choices, (T, k)
    int32_t *chosen;
    void *hidden;              // bf16 (experts, tp, F), experts = min(E, T k)
    void *out;
    int64_t ld_logits, ld_residual, ld_out;
    int T, H, F, E, k, normalize;
    bool bf16;                 // the logits
    FewShape shape;            // tp; the rest is set by the launch
};
cudaError_t launch_moe_few(MoeFewArgs a, int num_sms, const ErrCtx &err, cudaStream_t s);

}  // namespace tmg
