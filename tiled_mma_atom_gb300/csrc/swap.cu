// swap.cu — the bf16 instantiations of swap_kernel.cuh (swap_e4m3.cu holds
// the E4M3 ones, so that the two compile in parallel) and their dispatch.
#include "swap_kernel.cuh"

namespace tmg {

cudaError_t launch_swap_e4m3(const SwapArgs &a, int epi, int num_sms, const ErrCtx &err, cudaStream_t s);

cudaError_t launch_swap(const SwapArgs &a, int epi, bool e4m3, int num_sms, const ErrCtx &err, cudaStream_t s)
{
    if (e4m3)
        return launch_swap_e4m3(a, epi, num_sms, err, s);
    switch (epi) {
    case kSwPlain: return launch_swap_as<kInBf16, kSwPlain>(a, num_sms, err, s);
    case kSwDense: return launch_swap_as<kInBf16, kSwDense>(a, num_sms, err, s);
    case kSwSwiglu: return launch_swap_as<kInBf16, kSwSwiglu>(a, num_sms, err, s);
    default: return launch_swap_as<kInBf16, kSwSwigluGrad>(a, num_sms, err, s);
    }
}

}  // namespace tmg
