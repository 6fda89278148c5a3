// Linear attention, kernels of the gradients in __nv_bfloat16.
#include "linattn.cuh"

namespace gbfft {

cudaError_t attn_bf16_bwd(const AttnArgs& a, cudaStream_t s) { return attn_any<__nv_bfloat16, true>(a, FFT_BF16, s); }

}  // namespace gbfft
