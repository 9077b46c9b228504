// Forward pass over packed sequences of different lengths: instantiations of
// the kernel in fa_fwd_kernel.cuh that take their work from a plan.
#include "fa_fwd_kernel.cuh"

namespace fa {

cudaError_t launch_fwd_ragged(const FwdLaunch& a, cudaStream_t stream) {
  switch (a.d) {
    case 64:
      return a.causal ? launch_fwd_t<64, true, false, true>(a, stream) : launch_fwd_t<64, false, false, true>(a, stream);
    case 128:
      return a.causal ? launch_fwd_t<128, true, false, true>(a, stream) : launch_fwd_t<128, false, false, true>(a, stream);
    case 256:
      return a.causal ? launch_fwd_t<256, true, false, true>(a, stream) : launch_fwd_t<256, false, false, true>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fa
