// Linear attention, kernels of outputs in __nv_bfloat16.
#include "linattn.cuh"

namespace gbfft {

cudaError_t attn_bf16_fwd(const AttnArgs& a, cudaStream_t s) { return attn_any<__nv_bfloat16, false>(a, FFT_BF16, s); }

}  // namespace gbfft
