// wgrad.h — arguments of the grouped weight gradient's tensor-core kernel.
#pragma once

#include "internal.h"

namespace tmg {

constexpr int kWgCutBlocks = 22;    // cost of a tile's cut in blocks of 64 rows, two more for every piece

struct WgradTmaArgs {
    CUtensorMap tmD, tmA;      // dD (R, N) and A (R, K), boxes of 64 columns x 64 rows
    CUtensorMap tmD16, tmA16;  // the same, boxes of 16 rows
    CUtensorMap tmDg, tmAg;    // the same, boxes of one row (gathers)
    CUtensorMap tmOut;         // dB (E, N, K), boxes of 64 columns x 32 rows
    int tma_out;               // tmOut is there (16-byte rows)
    void *dB;                  // (E, N, K) contiguous
    const int32_t *offsets;
    int R, N, K, E;
    int group;                 // column tiles of dD per band
    int stages;                // set by the launch
    float *partials;           // wgrad_partial_bytes(); null: no tile is cut
    uint32_t *counters;        // 16 per cut tile
    uint32_t *feed;            // the tile counter
};
size_t wgrad_partial_bytes(int num_sms);
cudaError_t launch_wgrad(const WgradTmaArgs &a, int num_sms, const ErrCtx &err, cudaStream_t s);

}  // namespace tmg
