// Launches of the gated-scan kernels for one activation type: how many warps and CTAs share a
// slab of channels, and the template for it.
#pragma once

#include <algorithm>

#include "scan_kernels.cuh"

namespace gdnq {

struct ScanShape {
  int warps, tokens, cluster;  // template arguments W, T, CL
};

inline ScanShape scan_shape(int64_t units, int L) {
  if (L == 1) return {1, 1, 1};
  if (L <= 8 || units >= 2368) return {1, 8, 1};
  int cl = 1;
  while (cl < 8 && units * cl * kScanWarps < 1776 && cl * kScanWarps * 8 < L) cl *= 2;
  return {kScanWarps, 8, cl};
}

inline int scan_backward_cluster(int64_t units, int L) {
  int cl = 1;
  while (cl < 8 && units * cl * kScanWarps < 1776 && cl * GDN_SCAN_CHUNK < L) cl *= 2;
  return cl;
}

template <typename... Params>
cudaError_t launch_in_clusters(void (*kernel)(Params...), unsigned grid, int cluster,
                               cudaStream_t st, Params... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kScanWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = cluster > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename Act, int SCALE, int VEC>
cudaError_t launch_scan_vec(const ScanArgs& a, bool backward, cudaStream_t st) {
  const int slabs = (a.C + 32 * VEC - 1) / (32 * VEC);
  const int64_t units = (int64_t)a.B * slabs;
  if (backward) {
    const int cl = scan_backward_cluster(units, a.L);
    const unsigned grid = (unsigned)(units * cl);
    switch (cl) {
      case 1:
        return launch_in_clusters(scan_backward_kernel<Act, SCALE, VEC, 8, 8, 1>, grid, cl, st, a, slabs);
      case 2:
        return launch_in_clusters(scan_backward_kernel<Act, SCALE, VEC, 8, 8, 2>, grid, cl, st, a, slabs);
      case 4:
        return launch_in_clusters(scan_backward_kernel<Act, SCALE, VEC, 8, 8, 4>, grid, cl, st, a, slabs);
      default:
        return launch_in_clusters(scan_backward_kernel<Act, SCALE, VEC, 8, 8, 8>, grid, cl, st, a, slabs);
    }
  }
  const ScanShape s = scan_shape(units, a.L);
  const int groups = kScanWarps / s.warps;
  const unsigned grid =
      (unsigned)(s.cluster > 1 ? units * s.cluster : (units + groups - 1) / groups);
  if (s.tokens == 1)
    return launch_in_clusters(scan_kernel<Act, SCALE, VEC, 1, 1, 1>, grid, 1, st, a, slabs);
  if (s.warps == 1)
    return launch_in_clusters(scan_kernel<Act, SCALE, VEC, 1, 8, 1>, grid, 1, st, a, slabs);
  switch (s.cluster) {
    case 1:
      return launch_in_clusters(scan_kernel<Act, SCALE, VEC, 8, 8, 1>, grid, 1, st, a, slabs);
    case 2:
      return launch_in_clusters(scan_kernel<Act, SCALE, VEC, 8, 8, 2>, grid, 2, st, a, slabs);
    case 4:
      return launch_in_clusters(scan_kernel<Act, SCALE, VEC, 8, 8, 4>, grid, 4, st, a, slabs);
    default:
      return launch_in_clusters(scan_kernel<Act, SCALE, VEC, 8, 8, 8>, grid, 8, st, a, slabs);
  }
}

// Pairs of channels may be moved as one when every pair lies in one head and is aligned.
inline bool pairs(const Tok& t, int D, size_t elem) {
  return t.p == nullptr ||
         (D % 2 == 0 && t.sb % 2 == 0 && t.sl % 2 == 0 && t.sh % 2 == 0 &&
          reinterpret_cast<uintptr_t>(t.p) % (2 * elem) == 0);
}

template <typename Act, int SCALE>
cudaError_t launch_scan_scale(const ScanArgs& a, bool backward, cudaStream_t st) {
  bool two = pairs(a.x, a.D, sizeof(Act)) && pairs(a.g, a.D, 4);
  if (backward)
    two = two && pairs(a.grad_o, a.D, sizeof(Act)) && pairs(a.grad_x, a.D, sizeof(Act)) &&
          pairs(a.grad_g, a.D, 4);
  else
    two = two && pairs(a.o, a.D, sizeof(Act));
  return two ? launch_scan_vec<Act, SCALE, 2>(a, backward, st)
             : launch_scan_vec<Act, SCALE, 1>(a, backward, st);
}

template <typename Act>
cudaError_t launch_scan_as(const ScanArgs& a, int scale, bool backward, cudaStream_t st) {
  switch (scale) {
    case GDN_SCALE_COMPLEMENT:
      return launch_scan_scale<Act, GDN_SCALE_COMPLEMENT>(a, backward, st);
    case GDN_SCALE_SQRT:
      return launch_scan_scale<Act, GDN_SCALE_SQRT>(a, backward, st);
    default:
      return launch_scan_scale<Act, GDN_SCALE_NONE>(a, backward, st);
  }
}

}  // namespace gdnq
