// split.cu — the instantiations of split_kernel.cuh and their dispatch.
#include <atomic>

#include "split_kernel.cuh"

namespace tmg {

int split_clusters(int size)
{
    static std::atomic<int> known[64][4];          // by device and log2(size); 0: not asked yet
    int dev = 0;
    const int at = size == 1 ? 0 : size == 2 ? 1 : size == 4 ? 2 : 3;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return 0;
    int n = known[dev][at].load(std::memory_order_relaxed);
    if (n)
        return n;
    auto kern = split_kernel<kInBf16, kSwDense>;
    const int smem = 1024 + 196608 + kSplitBars;   // one CTA per SM, as launched
    if (ensure_smem_attr(reinterpret_cast<const void *>(kern), smem) != cudaSuccess)
        return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(size));
    cfg.blockDim = dim3(kSplitThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(size);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    known[dev][at].store(n, std::memory_order_relaxed);
    return n;
}

cudaError_t launch_split(const SplitArgs &a, int epi, bool e4m3, int cluster, int tiles, const ErrCtx &err, cudaStream_t s)
{
    switch (epi) {
    case kSwPlain:
        return e4m3 ? launch_split_as<kInE4m3, kSwPlain>(a, cluster, tiles, err, s)
                    : launch_split_as<kInBf16, kSwPlain>(a, cluster, tiles, err, s);
    case kSwDense:
        return e4m3 ? launch_split_as<kInE4m3, kSwDense>(a, cluster, tiles, err, s)
                    : launch_split_as<kInBf16, kSwDense>(a, cluster, tiles, err, s);
    case kSwSwiglu:
        return e4m3 ? launch_split_as<kInE4m3, kSwSwiglu>(a, cluster, tiles, err, s)
                    : launch_split_as<kInBf16, kSwSwiglu>(a, cluster, tiles, err, s);
    default:
        return e4m3 ? launch_split_as<kInE4m3, kSwSwigluGrad>(a, cluster, tiles, err, s)
                    : launch_split_as<kInBf16, kSwSwigluGrad>(a, cluster, tiles, err, s);
    }
}

}  // namespace tmg
