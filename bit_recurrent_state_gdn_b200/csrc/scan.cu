// Gated scan: launches of the kernels in scan_kernels.cuh.
#include "scan_kernels.cuh"

namespace gdnq {
namespace {

template <typename Act, int SCALE>
cudaError_t go(const ScanArgs& a, bool backward, cudaStream_t st) {
  const int64_t n = (int64_t)a.B * a.C;
  const unsigned grid = (unsigned)((n + 127) / 128);
  if (backward)
    scan_backward_kernel<Act, SCALE><<<grid, 128, 0, st>>>(a);
  else
    scan_kernel<Act, SCALE><<<grid, 128, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename Act>
cudaError_t by_scale(const ScanArgs& a, int scale, bool backward, cudaStream_t st) {
  switch (scale) {
    case GDN_SCALE_COMPLEMENT:
      return go<Act, GDN_SCALE_COMPLEMENT>(a, backward, st);
    case GDN_SCALE_SQRT:
      return go<Act, GDN_SCALE_SQRT>(a, backward, st);
    default:
      return go<Act, GDN_SCALE_NONE>(a, backward, st);
  }
}

cudaError_t by_type(const ScanArgs& a, const gdn_scan_config& cfg, bool backward,
                    cudaStream_t st) {
  return cfg.act_dtype == GDN_DTYPE_F32 ? by_scale<float>(a, cfg.scale, backward, st)
                                        : by_scale<__nv_bfloat16>(a, cfg.scale, backward, st);
}

}  // namespace

cudaError_t launch_scan(const ScanArgs& a, const gdn_scan_config& cfg, cudaStream_t st) {
  return by_type(a, cfg, false, st);
}

cudaError_t launch_scan_backward(const ScanArgs& a, const gdn_scan_config& cfg, cudaStream_t st) {
  return by_type(a, cfg, true, st);
}

}  // namespace gdnq
