// swap_e4m3.cu — the E4M3 instantiations of swap_kernel.cuh.
#include "swap_kernel.cuh"

namespace tmg {

cudaError_t launch_swap_e4m3(const SwapArgs &a, int epi, int num_sms, const ErrCtx &err, cudaStream_t s)
{
    switch (epi) {
    case kSwPlain: return launch_swap_as<kInE4m3, kSwPlain>(a, num_sms, err, s);
    case kSwDense: return launch_swap_as<kInE4m3, kSwDense>(a, num_sms, err, s);
    case kSwSwiglu: return launch_swap_as<kInE4m3, kSwSwiglu>(a, num_sms, err, s);
    default: return launch_swap_as<kInE4m3, kSwSwigluGrad>(a, num_sms, err, s);
    }
}

}  // namespace tmg
