// split.h — arguments of the product kernel that splits a tile's contraction
// over a cluster (split_kernel.cuh).
#pragma once

#include "grouped.h"

namespace tmg {

constexpr int kSplitMaxStages = 12;

struct SplitArgs {
    CUtensorMap tmW;           // K-major: 128 rows (SwiGLU: 64) of a K block; MN-major: 64 x 64
    CUtensorMap tmX;           // w rows of a K block; gather: one row
    void *D;
    const int32_t *offsets, *rows;
    ProductEpi epi;
    int64_t ldd;
    int R, T, N, K, E;         // N: output columns (F with SwiGLU)
    int half_rows;             // SwiGLU: rows of B before its up half
    int maj, gather, map_rows;
    int w;                     // rows of A per tile, a multiple of 16, at most 256
    int tmem_cols;             // a power of two, 32 .. 256
    int stages, stage_bytes, ring_bytes;     // the ring also holds the w x 128 fp32 partial tile
};

// Clusters of `size` CTAs that run at the same time on the current device (0
// where the query fails).
int split_clusters(int size);
cudaError_t launch_split(const SplitArgs &a, int epi, bool e4m3, int cluster, int tiles, const ErrCtx &err, cudaStream_t s);

}  // namespace tmg
