// Linear attention, kernels of outputs in __half.
#include "linattn.cuh"

namespace gbfft {

cudaError_t attn_f16_fwd(const AttnArgs& a, cudaStream_t s) { return attn_any<__half, false>(a, FFT_F16, s); }

}  // namespace gbfft
