// Selective state-space scan of f32 sequences, backward.
#include "scan_bwd.cuh"

namespace gbfft {

cudaError_t scan_backward_f32(const ScanBwdArgs& a, cudaStream_t s) {
    return scan_bwd_run<float>(a, s);
}

}  // namespace gbfft
