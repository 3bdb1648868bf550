// Group norm: launches of the kernels in norm_kernels.cuh.
#include <algorithm>

#include "norm_kernels.cuh"

namespace gdnq {

__global__ void __launch_bounds__(256) norm_reduce_kernel(NormArgs a, int parts) {
  __shared__ float2 sum[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t n = a.per_channel ? (int64_t)a.H * a.D : a.D;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float2 s = make_float2(0.0f, 0.0f);
  if (c < n) {
    // the partials of channel c: one per part (its head alone), or one per part and head
    const int d = (int)(c % a.D);
    const int64_t h0 = c / a.D, step = a.per_channel ? a.H : 1;
    const int64_t count = a.per_channel ? parts : (int64_t)parts * a.H;
    for (int64_t i = warp; i < count; i += 8) {
      const float* p = a.partials + (h0 + i * step) * 2 * a.D + d;
      s.x += p[0];
      s.y += p[a.D];
    }
  }
  sum[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < n) {
    for (int w = 1; w < 8; ++w) {
      s.x += sum[w][lane].x;
      s.y += sum[w][lane].y;
    }
    a.grad_w[c] = s.x;
    if (a.grad_bias) a.grad_bias[c] = s.y;
  }
}

namespace {

constexpr int kSms = 148;

int backward_parts(int B, int L, int H) {
  return (int)std::max<int64_t>(1, std::min<int64_t>((int64_t)B * L, kSms * 8 / std::max(H, 1)));
}

template <typename Act, int NI>
cudaError_t go(const NormArgs& a, bool backward, cudaStream_t st) {
  if (!backward) {
    const int64_t rows = (int64_t)a.B * a.L * a.H;
    norm_kernel<Act, NI><<<(unsigned)std::min<int64_t>(rows, kSms * 64), kNormThreads, 0, st>>>(a);
    return cudaGetLastError();
  }
  const int parts = backward_parts(a.B, a.L, a.H);
  norm_backward_kernel<Act, NI><<<(unsigned)parts * (unsigned)a.H, kNormThreads, 0, st>>>(a, parts);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t n = a.per_channel ? (int64_t)a.H * a.D : a.D;
  norm_reduce_kernel<<<(unsigned)((n + 31) / 32), 256, 0, st>>>(a, parts);
  return cudaGetLastError();
}

template <typename Act>
cudaError_t by_size(const NormArgs& a, bool backward, cudaStream_t st) {
  if (a.D <= 256) return go<Act, 1>(a, backward, st);
  if (a.D <= 1024) return go<Act, 4>(a, backward, st);
  if (a.D <= 4096) return go<Act, 16>(a, backward, st);
  return go<Act, 32>(a, backward, st);
}

cudaError_t by_type(const NormArgs& a, const gdn_norm_config& cfg, bool backward,
                    cudaStream_t st) {
  return cfg.act_dtype == GDN_DTYPE_F32 ? by_size<float>(a, backward, st)
                                        : by_size<__nv_bfloat16>(a, backward, st);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, const gdn_norm_config& cfg, cudaStream_t st) {
  return by_type(a, cfg, false, st);
}

cudaError_t launch_norm_backward(const NormArgs& a, const gdn_norm_config& cfg, cudaStream_t st) {
  return by_type(a, cfg, true, st);
}

size_t norm_backward_workspace(const gdn_norm_config& cfg, int L) {
  return (size_t)backward_parts(cfg.B, L, cfg.H) * (size_t)cfg.H * 2 * (size_t)cfg.D * sizeof(float);
}

}  // namespace gdnq
