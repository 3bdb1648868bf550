// Group norm with f32 activations.
#include "norm_launch.cuh"

namespace gdnq {

cudaError_t launch_norm_f32(const NormArgs& a, bool backward, cudaStream_t st) {
  return launch_norm_as<float>(a, backward, st);
}

}  // namespace gdnq
