// Selective state-space scan of f16 sequences, forward.
#include "scan.cuh"

namespace gbfft {

cudaError_t scan_forward_f16(const ScanArgs& a, cudaStream_t s) {
    return scan_run<__half, SCAN_OUTPUT>(a, s);
}

}  // namespace gbfft
