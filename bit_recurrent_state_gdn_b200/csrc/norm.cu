// Group norm: the parameters' gradients from partial sums, and the workspace for them.
#include "norm_launch.cuh"

namespace gdnq {
namespace {

// grad_w and grad_bias from partials[count][2][D] (per head and channel: [parts][H][2][D]): a CTA
// takes 32 channels, its 32 warps every 32nd partial sum, added in the same order every time.
__global__ void __launch_bounds__(1024) norm_reduce_kernel(NormArgs a, int64_t count) {
  __shared__ float2 sum[32][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t n = a.per_channel ? (int64_t)a.H * a.D : a.D;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float2 s = make_float2(0.0f, 0.0f);
  wait_for_last();
  if (c < n) {
    const int64_t step = a.per_channel ? a.H : 1;
    const float* p = a.partials + c / a.D * 2 * a.D + c % a.D;
    for (int64_t i = warp * step; i < count; i += 32 * step) {
      s.x += p[i * 2 * a.D];
      s.y += p[i * 2 * a.D + a.D];
    }
  }
  sum[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < n) {
    for (int w = 1; w < 32; ++w) {
      s.x += sum[w][lane].x;
      s.y += sum[w][lane].y;
    }
    a.grad_w[c] = s.x;
    if (a.grad_bias) a.grad_bias[c] = s.y;
  }
}

}  // namespace

cudaError_t launch_norm_reduce(const NormArgs& a, int64_t partials, cudaStream_t st) {
  const int64_t n = a.per_channel ? (int64_t)a.H * a.D : a.D;
  return launch_behind(norm_reduce_kernel, (unsigned)((n + 31) / 32), 1024, st, a, partials);
}

// Large enough for any placement of the arrays, on which the split of the rows depends.
size_t norm_backward_workspace(const gdn_norm_config& cfg, int L) {
  const int64_t tokens = (int64_t)cfg.B * L;
  const bool per_channel = cfg.weight == GDN_WEIGHT_CHANNEL;
  int64_t most = (int64_t)norm_wide_parts(tokens, cfg.H) * cfg.H;
  if (cfg.D <= kNormWarp) {
    const int elem = cfg.act_dtype == GDN_DTYPE_F32 ? 4 : 2;
    // for either number of CTAs per SM: fewer of them may take more parts (shares is not monotonic)
    for (const int resident : {norm_resident(8, true), norm_resident(16, true)})
      for (int lanes = 2; lanes <= 32; lanes *= 2)
        most = std::max(most, norm_partials(norm_plan(cfg.D, cfg.H, tokens, elem, lanes, resident), cfg.H,
                                            per_channel));
  }
  return (size_t)most * 2 * (size_t)cfg.D * sizeof(float);
}

}  // namespace gdnq
