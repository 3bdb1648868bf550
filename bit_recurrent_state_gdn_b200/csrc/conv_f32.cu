// Short convolution with f32 activations.
#include "conv_launch.cuh"

namespace gdnq {

cudaError_t launch_conv_f32(const ConvArgs& a, bool backward, cudaStream_t st) {
  return launch_conv_as<float>(a, backward, st);
}

}  // namespace gdnq
