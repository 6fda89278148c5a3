// Selective state-space scan of bf16 sequences, backward.
#include "scan_bwd.cuh"

namespace gbfft {

cudaError_t scan_backward_bf16(const ScanBwdArgs& a, cudaStream_t s) {
    return scan_bwd_run<__nv_bfloat16>(a, s);
}

}  // namespace gbfft
