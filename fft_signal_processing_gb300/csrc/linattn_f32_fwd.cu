// Linear attention, kernels of outputs in float.
#include "linattn.cuh"

namespace gbfft {

cudaError_t attn_f32_fwd(const AttnArgs& a, cudaStream_t s) { return attn_any<float, false>(a, FFT_F32, s); }

}  // namespace gbfft
