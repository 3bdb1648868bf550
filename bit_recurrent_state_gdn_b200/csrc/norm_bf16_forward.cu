// Group norm with bf16 activations, forward.
#include "norm_launch.cuh"

namespace gdnq {

cudaError_t launch_norm_bf16_forward(const NormArgs& a, cudaStream_t st) {
  return launch_norm_as<__nv_bfloat16, false>(a, st);
}

}  // namespace gdnq
