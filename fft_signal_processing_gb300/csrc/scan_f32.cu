// Selective state-space scan of f32 sequences, forward.
#include "scan.cuh"

namespace gbfft {

cudaError_t scan_forward_f32(const ScanArgs& a, cudaStream_t s) {
    return scan_run<float, SCAN_OUTPUT>(a, s);
}

}  // namespace gbfft
