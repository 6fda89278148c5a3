// Linear attention, kernels of the gradients in float.
#include "linattn.cuh"

namespace gbfft {

cudaError_t attn_f32_bwd(const AttnArgs& a, cudaStream_t s) { return attn_any<float, true>(a, FFT_F32, s); }

}  // namespace gbfft
