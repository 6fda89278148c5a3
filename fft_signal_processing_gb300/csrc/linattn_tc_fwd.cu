// Linear attention on tcgen05, kernels of outputs in bfloat16.
#include "linattn_tc.cuh"

namespace gbfft {

cudaError_t attn_tc_fwd(const AttnArgs& a, int* err, cudaStream_t s) {
    if (a.dx <= 64) return a.dz <= 64 ? launch_attn_tc<64, 64, false>(a, err, s) : launch_attn_tc<64, 128, false>(a, err, s);
    return a.dz <= 64 ? launch_attn_tc<128, 64, false>(a, err, s) : launch_attn_tc<128, 128, false>(a, err, s);
}

}  // namespace gbfft
