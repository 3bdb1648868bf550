// Short convolution with bf16 activations.
#include "conv_launch.cuh"

namespace gdnq {

cudaError_t launch_conv_bf16(const ConvArgs& a, bool backward, cudaStream_t st) {
  return launch_conv_as<__nv_bfloat16>(a, backward, st);
}

}  // namespace gdnq
