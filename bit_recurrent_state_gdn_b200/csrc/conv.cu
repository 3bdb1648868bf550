// Short convolution: launches of the kernels in conv_kernels.cuh.
#include <algorithm>

#include "conv_kernels.cuh"

namespace gdnq {
namespace {

constexpr int kSms = 148;

int conv_runs(int L) { return std::max(1, (int)(((int64_t)L + kConvRun - 1) / kConvRun)); }
int conv_slabs(int C) { return (C + 31) / 32; }
int conv_parts(int B, int L, int C) {
  const int64_t runs = (int64_t)B * conv_runs(L);
  return (int)std::max<int64_t>(1, std::min<int64_t>((runs + 7) / 8, kSms * 8 / conv_slabs(C)));
}

template <typename Act, int K>
cudaError_t go(const ConvArgs& a, bool backward, cudaStream_t st) {
  const int runs = conv_runs(a.L);
  if (!backward) {
    const int64_t n = (int64_t)a.B * runs * a.C;
    conv_kernel<Act, K><<<(unsigned)((n + 255) / 256), 256, 0, st>>>(a, runs);
    return cudaGetLastError();
  }
  const int slabs = conv_slabs(a.C), parts = conv_parts(a.B, a.L, a.C);
  conv_backward_kernel<Act, K><<<(unsigned)(slabs * parts), 256, 0, st>>>(a, runs, slabs);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t n = (int64_t)a.C * (K + 1);
  conv_reduce_kernel<K><<<(unsigned)((n + 127) / 128), 128, 0, st>>>(a, parts);
  return cudaGetLastError();
}

template <typename Act>
cudaError_t by_taps(const ConvArgs& a, bool backward, cudaStream_t st) {
  switch (a.K) {
    case 2:
      return go<Act, 2>(a, backward, st);
    case 3:
      return go<Act, 3>(a, backward, st);
    default:
      return go<Act, 4>(a, backward, st);
  }
}

cudaError_t by_type(const ConvArgs& a, const gdn_conv_config& cfg, bool backward,
                    cudaStream_t st) {
  return cfg.act_dtype == GDN_DTYPE_F32 ? by_taps<float>(a, backward, st)
                                        : by_taps<__nv_bfloat16>(a, backward, st);
}

}  // namespace

cudaError_t launch_conv(const ConvArgs& a, const gdn_conv_config& cfg, cudaStream_t st) {
  return by_type(a, cfg, false, st);
}

cudaError_t launch_conv_backward(const ConvArgs& a, const gdn_conv_config& cfg, cudaStream_t st) {
  return by_type(a, cfg, true, st);
}

size_t conv_backward_workspace(const gdn_conv_config& cfg, int L) {
  const int C = cfg.H * cfg.D;
  return (size_t)conv_parts(cfg.B, L, C) * (size_t)C * (size_t)(cfg.K + 1) * sizeof(float);
}

}  // namespace gdnq
