// Group norm with bf16 activations.
#include "norm_launch.cuh"

namespace gdnq {

cudaError_t launch_norm_bf16(const NormArgs& a, bool backward, cudaStream_t st) {
  return launch_norm_as<__nv_bfloat16>(a, backward, st);
}

}  // namespace gdnq
