// Group norm with f32 activations, backward.
#include "norm_launch.cuh"

namespace gdnq {

cudaError_t launch_norm_f32_backward(const NormArgs& a, cudaStream_t st) {
  return launch_norm_as<float, true>(a, st);
}

}  // namespace gdnq
