// Group norm with f32 activations, forward.
#include "norm_launch.cuh"

namespace gdnq {

cudaError_t launch_norm_f32_forward(const NormArgs& a, cudaStream_t st) {
  return launch_norm_as<float, false>(a, st);
}

}  // namespace gdnq
