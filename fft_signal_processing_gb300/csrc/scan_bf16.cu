// Selective state-space scan of bf16 sequences, forward.
#include "scan.cuh"

namespace gbfft {

cudaError_t scan_forward_bf16(const ScanArgs& a, cudaStream_t s) {
    return scan_run<__nv_bfloat16, SCAN_OUTPUT>(a, s);
}

}  // namespace gbfft
