// Selective state-space scan of f16 sequences, backward.
#include "scan_bwd.cuh"

namespace gbfft {

cudaError_t scan_backward_f16(const ScanBwdArgs& a, cudaStream_t s) {
    return scan_bwd_run<__half>(a, s);
}

}  // namespace gbfft
