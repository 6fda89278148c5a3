// Linear attention, kernels of the gradients in __half.
#include "linattn.cuh"

namespace gbfft {

cudaError_t attn_f16_bwd(const AttnArgs& a, cudaStream_t s) { return attn_any<__half, true>(a, FFT_F16, s); }

}  // namespace gbfft
