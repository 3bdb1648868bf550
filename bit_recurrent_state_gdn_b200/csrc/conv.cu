// Short convolution: the parameters' gradients from partial sums, and the workspace for them.
#include "conv_launch.cuh"

namespace gdnq {
namespace {

// grad_w [C][K] and grad_bias [C] from partials[parts][K + 1][C]: a CTA takes 32 sums, its 8
// warps every 8th part, added in the same order every time.
__global__ void __launch_bounds__(256) conv_reduce_kernel(ConvArgs a, int parts) {
  __shared__ float sum[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t n = (int64_t)a.C * (a.K + 1), i = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.0f;
  wait_for_last();
  if (i < n)
    for (int p = warp; p < parts; p += 8) s += a.partials[p * n + i];
  sum[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && i < n) {
    for (int w = 1; w < 8; ++w) s += sum[w][lane];
    const int64_t c = i % a.C;
    const int j = (int)(i / a.C);
    if (j < a.K)
      a.grad_w[c * a.K + j] = s;
    else if (a.grad_bias)
      a.grad_bias[c] = s;
  }
}

}  // namespace

cudaError_t launch_conv_reduce(const ConvArgs& a, int parts, cudaStream_t st) {
  const int64_t n = (int64_t)a.C * (a.K + 1);
  return launch_behind(conv_reduce_kernel, (unsigned)((n + 31) / 32), 256, st, a, parts);
}

// Large enough for any placement of the arrays, on which the split depends.
size_t conv_backward_workspace(const gdn_conv_config& cfg, int L) {
  const int C = cfg.H * cfg.D;
  int parts = 1;
  for (const int V : {1, 2, kConvBackVec}) parts = std::max(parts, conv_backward_split(cfg.B, L, C, V).parts);
  return (size_t)parts * (size_t)C * (size_t)(cfg.K + 1) * sizeof(float);
}

}  // namespace gdnq
