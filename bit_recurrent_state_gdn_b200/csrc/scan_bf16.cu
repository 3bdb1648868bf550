// Gated scan with bf16 activations.
#include "scan_launch.cuh"

namespace gdnq {

cudaError_t launch_scan_bf16(const ScanArgs& a, int scale, bool backward, cudaStream_t st) {
  return launch_scan_as<__nv_bfloat16>(a, scale, backward, st);
}

}  // namespace gdnq
