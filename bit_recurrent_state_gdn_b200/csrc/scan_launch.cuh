// Launches of the gated-scan kernels for one activation type: how many warps and CTAs share a
// slab of channels, and the template for it.
#pragma once

#include <algorithm>

#include "scan_kernels.cuh"
#include "window_dispatch.cuh"
namespace gdnq {

template <typename... Params>
cudaError_t launch_in_clusters(void (*kernel)(Params...), int64_t grid, int threads, int cluster,
                               int shared, cudaStream_t st, Params... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)shared;
  cfg.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = cluster > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename Act, int SCALE, class Runs, int W, int CL, int MINB>
cudaError_t scan_forward(const ScanArgs& a, int slabs, cudaStream_t st) {
  constexpr auto kernel = scan_kernel<Act, SCALE, Runs, W, CL, MINB>;
  constexpr int kThreads = scan_threads(W), kShared = kThreads / 32 * Runs::kBytes;
  // above 48 KB the limit has to be raised, and the joins' static arrays count too
  const cudaError_t e = ensure_smem<kernel>(kShared ? std::max(kShared, 48 * 1024 + 16) : 0);
  if (e != cudaSuccess) return e;
  const int64_t units = (int64_t)a.B * slabs;
  const int64_t grid = (units + scan_groups(W) - 1) / scan_groups(W) * CL;
  return launch_in_clusters(kernel, grid, kThreads, CL, kShared, st, a, slabs);
}

template <typename Act, int SCALE, class Runs, int W, int CL, int MINB>
cudaError_t scan_back(const ScanArgs& a, int slabs, cudaStream_t st) {
  constexpr auto kernel = scan_backward_kernel<Act, SCALE, Runs, W, CL, MINB>;
  constexpr int kThreads = scan_threads(W), kShared = kThreads / 32 * Runs::kBytes;
  const cudaError_t e = ensure_smem<kernel>(kShared ? std::max(kShared, 48 * 1024 + 16) : 0);
  if (e != cudaSuccess) return e;
  const int64_t units = (int64_t)a.B * slabs;
  const int64_t grid = (units + scan_groups(W) - 1) / scan_groups(W) * CL;
  return launch_in_clusters(kernel, grid, kThreads, CL, kShared, st, a, slabs);
}

// CTAs that share a unit (a slab of channels of one sequence) as a cluster: where units are
// few, as many as two CTAs per SM hold, each with a tile of its own to take.
inline int scan_cluster(int64_t units, int tile, int L) {
  int cl = 1;
  while (cl < 8 && units * cl * 2 <= 296 && cl * tile < L) cl *= 2;
  return cl;
}

// How a forward scan shares its units out. Measured on 64 units per sequence, bf16, in GB/s of
// 6452 (four warps a unit and four CTAs per SM / eight and two):
//   64 units  2305 / 2833, clusters of four CTAs of eight 4670    128  3973 / 5365
//   256  5750 / 6074    384  6209 / 5674    512  6415 / 6006    768  5360 / 5953
//   1024  6149 / 6368   1280  5994 / 6183   1664  6405 / 5938   2560  6337 / 5824
// so: eight warps where they fit at once or where four leave a second wave half empty. Units of
// few tokens go to one warp each, eight units a CTA, without joins: 2048 units of 100 tokens 5299
// against 4248 with four warps, 16384 of 64 tokens 6225 / 4803, 4096 of 512 tokens 6335 / 6571.
enum class ScanSplit { Alone, Four, Eight };

inline ScanSplit scan_split(int64_t units, int L, int run) {
  if (L <= run || (units >= 2048 && L <= 256)) return ScanSplit::Alone;
  return (units > 296 && units <= 592) || units > 1480 ? ScanSplit::Four : ScanSplit::Eight;
}

// The two kernels of sequences split into spans.
template <typename Act, int SCALE, class P>
cudaError_t launch_scan_split(ScanArgs a, bool backward, int slabs, cudaStream_t st) {
  using Span = typename P::Alone;
  const int64_t grid = (int64_t)a.B * slabs * a.spans_per_unit;
  constexpr int kSpanShared = 8 * Span::kBytes;
  constexpr int kRaised = kSpanShared ? std::max(kSpanShared, 48 * 1024 + 16) : 0;
  if (backward) {
    constexpr auto spans = scan_span_kernel<Act, SCALE, Span, true>;
    cudaError_t e = ensure_smem<spans>(kRaised);
    ScanArgs over = a;
    over.x = a.grad_o;
    if (e == cudaSuccess) e = launch_in_clusters(spans, grid, 256, 1, kSpanShared, st, over, slabs);
    if (e != cudaSuccess) return e;
    using Back = typename P::Back;
    constexpr int W = GDN_SCAN_CHUNK / Back::kTokens, kShared = W * Back::kBytes;
    constexpr auto kernel = scan_backward_kernel<Act, SCALE, Back, W, 1, P::kBackResident, true>;
    e = ensure_smem<kernel>(kShared ? std::max(kShared, 48 * 1024 + 16) : 0);
    return e == cudaSuccess ? launch_in_clusters(kernel, grid, 32 * W, 1, kShared, st, a, slabs) : e;
  }
  constexpr auto spans = scan_span_kernel<Act, SCALE, Span, false>;
  cudaError_t e = ensure_smem<spans>(kRaised);
  if (e == cudaSuccess) e = launch_in_clusters(spans, grid, 256, 1, kSpanShared, st, a, slabs);
  if (e != cudaSuccess) return e;
  using Eight = typename P::Eight;
  constexpr int kShared = 8 * Eight::kBytes;
  constexpr auto kernel = scan_kernel<Act, SCALE, Eight, 8, 1, 2, true>;
  e = ensure_smem<kernel>(kShared ? std::max(kShared, 48 * 1024 + 16) : 0);
  return e == cudaSuccess ? launch_in_clusters(kernel, grid, 256, 1, kShared, st, a, slabs) : e;
}

template <typename Act, int SCALE, class P>
cudaError_t launch_scan_plan(const ScanArgs& a, bool backward, cudaStream_t st) {
  const int slabs = (a.C + kScanSlab - 1) / kScanSlab;
  const int64_t units = (int64_t)a.B * slabs;
  if (a.spans) return launch_scan_split<Act, SCALE, P>(a, backward, slabs, st);
  if (backward) {
    // sequences of one run need no joins (52 x 2150 channels, 1 token: 35 us with a CTA each)
    if (a.L <= P::BackAlone::kTokens)
      return scan_back<Act, SCALE, typename P::BackAlone, 1, 1, 1>(a, slabs, st);
    using Back = typename P::Back;
    constexpr int W = GDN_SCAN_CHUNK / Back::kTokens, kResident = P::kBackResident;
    switch (scan_cluster(units, GDN_SCAN_CHUNK, a.L)) {
      case 1:
        return scan_back<Act, SCALE, Back, W, 1, kResident>(a, slabs, st);
      case 2:
        return scan_back<Act, SCALE, Back, W, 2, kResident>(a, slabs, st);
      case 4:
        return scan_back<Act, SCALE, Back, W, 4, kResident>(a, slabs, st);
      default:
        return scan_back<Act, SCALE, Back, W, 8, kResident>(a, slabs, st);
    }
  }
  if (a.L <= 1) return scan_forward<Act, SCALE, typename P::One, 1, 1, 4>(a, slabs, st);
  switch (scan_split(units, a.L, P::Alone::kTokens)) {
    case ScanSplit::Alone:
      return scan_forward<Act, SCALE, typename P::Alone, 1, 1, 2>(a, slabs, st);
    case ScanSplit::Four:
      return scan_forward<Act, SCALE, typename P::Four, 4, 1, 4>(a, slabs, st);
    default:
      break;
  }
  using Eight = typename P::Eight;
  switch (scan_cluster(units, 8 * Eight::kTokens, a.L)) {
    case 8:
      return scan_forward<Act, SCALE, Eight, 8, 8, 2>(a, slabs, st);
    case 4:
      return scan_forward<Act, SCALE, Eight, 8, 4, 2>(a, slabs, st);
    default:  // two CTAs of a cluster gain nothing over one (128 units: 4994 / 5365 GB/s)
      return scan_forward<Act, SCALE, Eight, 8, 1, 2>(a, slabs, st);
  }
}

// Rows that 16-byte pieces cover. Runs of 16 tokens against 8 halve the joins (512 units of 4096
// tokens: 167 / 185 us); two stages of them keep as many bytes in flight as four of 8. Eight warps
// of fp32 rows would fill an SM's shared memory with one CTA, so theirs are runs of 8.
template <typename Act>
struct PlanShared {
  static constexpr bool kF32 = sizeof(Act) == 4;
  using One = RunsInRegisters<Act, 1, 1, false>;
  using Alone = RunsInShared<Act, 8, 4, false>;
  using Four = RunsInShared<Act, 16, 2, false>;
  using Eight = RunsInShared<Act, kF32 ? 8 : 16, kF32 ? 3 : 2, false>;
  using Back = RunsInShared<Act, 16, 2, true>;
  using BackAlone = RunsInRegisters<Act, 1, 8, true>;
  static constexpr int kBackResident = 2;
};

// Any other placement: neighbouring channels (STEP = 1), or one by one (32).
template <typename Act, int STEP>
struct PlanRegisters {
  using One = RunsInRegisters<Act, STEP, 1, false>;
  using Alone = RunsInRegisters<Act, STEP, 8, false>;
  using Four = Alone;
  using Eight = Alone;
  using Back = RunsInRegisters<Act, STEP, 8, true>;
  using BackAlone = Back;
  static constexpr int kBackResident = 1;  // two spill (3875 channels, 8 x 1000 tokens: 1.5 / 2.2 TB/s)
};

// Whether `n` channels may be moved as one in every array: they lie in one head and are aligned.
inline bool aligned(const Tok& t, int D, int n, size_t elem) {
  return D % n == 0 && t.sb % n == 0 && t.sl % n == 0 && t.sh % n == 0 &&
         reinterpret_cast<uintptr_t>(t.p) % (n * elem) == 0;
}

template <typename Act, int SCALE>
cudaError_t launch_scan_scale(ScanArgs a, bool backward, cudaStream_t st) {
  struct Used {
    const Tok* t;
    size_t elem;
  };
  const Used read[3] = {{&a.x, sizeof(Act)}, {&a.g, 4}, {backward ? &a.grad_o : &a.x, sizeof(Act)}};
  const Used written[2] = {{backward ? &a.grad_x : &a.o, sizeof(Act)},
                           {backward ? &a.grad_g : &a.o, backward ? 4 : sizeof(Act)}};
  // where a token's heads follow one another in every array, they are one head of C channels
  bool dense = true;
  for (const Used& u : read) dense = dense && u.t->sh == a.D;
  for (const Used& u : written) dense = dense && u.t->sh == a.D;
  if (dense || a.H == 1) {
    a.D = a.C;
    a.H = 1;
    a.x.sh = a.g.sh = a.o.sh = a.grad_o.sh = a.grad_x.sh = a.grad_g.sh = 0;
  }
  bool pairs = true, pieces = a.L > 0;
  for (const Used& u : read) {
    pairs = pairs && aligned(*u.t, a.D, 2, u.elem);
    pieces = pieces && aligned(*u.t, a.D, (int)(16 / u.elem), u.elem);
  }
  for (const Used& u : written) pairs = pairs && aligned(*u.t, a.D, 2, u.elem);
  // 16-byte pieces, channel pairs, single channels
  if (pairs && pieces) return launch_scan_plan<Act, SCALE, PlanShared<Act>>(a, backward, st);
  if (pairs) return launch_scan_plan<Act, SCALE, PlanRegisters<Act, 1>>(a, backward, st);
  return launch_scan_plan<Act, SCALE, PlanRegisters<Act, 32>>(a, backward, st);
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
