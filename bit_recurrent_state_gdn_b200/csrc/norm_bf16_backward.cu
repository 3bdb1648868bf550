// Group norm with bf16 activations, backward.
#include "norm_launch.cuh"

namespace gdnq {

cudaError_t launch_norm_bf16_backward(const NormArgs& a, cudaStream_t st) {
  return launch_norm_as<__nv_bfloat16, true>(a, st);
}

}  // namespace gdnq
