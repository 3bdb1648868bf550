// Gated scan with fp32 activations.
#include "scan_launch.cuh"

namespace gdnq {

cudaError_t launch_scan_f32(const ScanArgs& a, int scale, bool backward, cudaStream_t st) {
  return launch_scan_as<float>(a, scale, backward, st);
}

}  // namespace gdnq
