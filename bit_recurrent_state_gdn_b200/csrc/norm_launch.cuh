// Launches of the group-norm kernels for one activation type.
#pragma once

#include <algorithm>

#include "norm_kernels.cuh"
#include "window_dispatch.cuh"

namespace gdnq {

// The lanes of a row, the heads of a CTA and the CTAs of a launch. Heads side by side make a
// token's reads at least 512 bytes long where the heads allow it without idle lanes, and 128 with
// them.
inline NormSplit norm_plan(int D, int H, int64_t tokens, int elem, int lanes, int resident) {
  NormSplit s;
  s.lanes = lanes;
  const int rows = kNormThreads / lanes;
  int hb = 1, log = 0;
  while (hb * 2 <= rows && ((H % (hb * 2) == 0 && hb * D * elem < 512) ||
                            (hb < H && hb * D * elem < 128)))
    hb *= 2, ++log;
  s.hb_log = log;
  s.heads_of_blocks = (H + hb - 1) / hb;
  const int64_t tb = rows / hb, most = (tokens + tb - 1) / tb;
  s.parts = (int)std::max<int64_t>(1, std::min<int64_t>(most, shares(kSms * resident, s.heads_of_blocks)));
  return s;
}

// Lanes for `pieces` of them per row (ring or single elements).
inline int norm_lanes(int pieces, int fewest) {
  int lanes = fewest;
  while (lanes < 32 && lanes < pieces) lanes *= 2;
  return lanes;
}

constexpr int kNormWide = 1024;  // channels of a head that a warp holds

inline int norm_wide_parts(int64_t tokens, int H) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(tokens, kSms * 8 / std::max(H, 1)));
}

// Partial sums of a launch: their number, for each D (or H D) channels.
inline int64_t norm_partials(const NormSplit& s, int H, bool per_channel) {
  return per_channel ? (int64_t)s.parts * H : (int64_t)s.parts * s.heads_of_blocks;
}

cudaError_t launch_norm_reduce(const NormArgs& a, int64_t partials, cudaStream_t st);

// CTAs per SM that the kernels' registers are bounded for, by the channels that a lane holds. With
// eight, four forward (152 us against 139, 8 x 32 x 4096 gated rows of 128) and three backward
// (188 us against 118, four sequences) spill.
constexpr int norm_resident(int channels, bool backward) {
  return backward ? (channels <= 16 ? 2 : 1) : (channels <= 8 ? 3 : 2);
}

template <typename Act, bool GATE, class F, class B>
cudaError_t norm_go(const NormArgs& a, bool backward, cudaStream_t st) {
  const int64_t tokens = (int64_t)a.B * a.L;
  if (!backward) {
    constexpr int kResident = norm_resident(F::NI * F::V, false);
    constexpr auto kernel = norm_kernel<Act, GATE, F, kResident>;
    cudaError_t e = ensure_smem<kernel>(F::kBytes);
    if (e != cudaSuccess) return e;
    const NormSplit s = norm_plan(a.D, a.H, tokens, sizeof(Act), F::LANES, kResident);
    kernel<<<(unsigned)s.parts * (unsigned)s.heads_of_blocks, kNormThreads, F::kBytes, st>>>(a, s);
    return cudaGetLastError();
  }
  constexpr int kResident = norm_resident(B::NI * B::V, true);
  constexpr auto kernel = norm_backward_kernel<Act, GATE, B, kResident>;
  constexpr int kShared = norm_backward_shared<B>();
  cudaError_t e = ensure_smem<kernel>(kShared);
  if (e != cudaSuccess) return e;
  const NormSplit s = norm_plan(a.D, a.H, tokens, sizeof(Act), B::LANES, kResident);
  kernel<<<(unsigned)s.parts * (unsigned)s.heads_of_blocks, kNormThreads, kShared, st>>>(a, s);
  e = cudaGetLastError();
  return e == cudaSuccess ? launch_norm_reduce(a, norm_partials(s, a.H, a.per_channel), st) : e;
}

template <typename Act, bool GATE, int LANES, int NI>
cudaError_t norm_ring(const NormArgs& a, bool backward, cudaStream_t st) {
  constexpr int kF = GATE ? 2 : 1, kB = kF + 1;
  return norm_go<Act, GATE, PiecesInShared<Act, LANES, NI, kF, NI <= 2 ? 4 : NI == 4 ? 3 : 2>,
                 PiecesInShared<Act, LANES, NI, kB, NI == 1 ? 4 : NI == 2 ? 3 : 2>>(a, backward, st);
}

template <typename Act, bool GATE, int LANES, int NI>
cudaError_t norm_direct(const NormArgs& a, bool backward, cudaStream_t st) {
  constexpr int kF = GATE ? 2 : 1;
  return norm_go<Act, GATE, PiecesInRegisters<Act, LANES, NI, kF>,
                 PiecesInRegisters<Act, LANES, NI, kF + 1>>(a, backward, st);
}

template <typename Act, int NI>
cudaError_t norm_wide(const NormArgs& a, bool backward, cudaStream_t st) {
  const int64_t tokens = (int64_t)a.B * a.L;
  if (!backward) {
    norm_wide_kernel<Act, NI><<<(unsigned)std::min<int64_t>(tokens * a.H, kSms * 8), kNormThreads, 0, st>>>(a);
    return cudaGetLastError();
  }
  const int parts = norm_wide_parts(tokens, a.H);
  norm_wide_backward_kernel<Act, NI><<<(unsigned)parts * (unsigned)a.H, kNormThreads, 0, st>>>(a, parts);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? launch_norm_reduce(a, (int64_t)parts * a.H, st) : e;
}

template <typename Act, bool GATE>
cudaError_t norm_by_size(const NormArgs& a, bool backward, bool pieces, cudaStream_t st) {
  if (a.D > kNormWide) {
    if (a.D <= 2048) return norm_wide<Act, 8>(a, backward, st);
    if (a.D <= 4096) return norm_wide<Act, 16>(a, backward, st);
    return norm_wide<Act, 32>(a, backward, st);
  }
  constexpr int V = 16 / (int)sizeof(Act);
  if (pieces) {
    const int n = a.D / V;
    switch (norm_lanes(n, 4)) {
      case 4:
        return norm_ring<Act, GATE, 4, 1>(a, backward, st);
      case 8:
        return norm_ring<Act, GATE, 8, 1>(a, backward, st);
      case 16:
        return norm_ring<Act, GATE, 16, 1>(a, backward, st);
      default:
        break;
    }
    if (n <= 32) return norm_ring<Act, GATE, 32, 1>(a, backward, st);
    if (n <= 64) return norm_ring<Act, GATE, 32, 2>(a, backward, st);
    if (n <= 128) return norm_ring<Act, GATE, 32, 4>(a, backward, st);
    if constexpr (V == 4) return norm_ring<Act, GATE, 32, 8>(a, backward, st);
  }
  if (a.D <= 8) return norm_direct<Act, GATE, 8, 1>(a, backward, st);
  if (a.D <= 32) return norm_direct<Act, GATE, 32, 1>(a, backward, st);
  if (a.D <= 64) return norm_direct<Act, GATE, 32, 2>(a, backward, st);
  if (a.D <= 128) return norm_direct<Act, GATE, 32, 4>(a, backward, st);
  if (a.D <= 256) return norm_direct<Act, GATE, 32, 8>(a, backward, st);
  if (a.D <= 512) return norm_direct<Act, GATE, 32, 16>(a, backward, st);
  return norm_direct<Act, GATE, 32, 32>(a, backward, st);
}

template <typename Act>
cudaError_t launch_norm_as(const NormArgs& a, bool backward, cudaStream_t st) {
  constexpr int V = 16 / (int)sizeof(Act);
  const Tok* used[5] = {&a.x, &a.z, backward ? &a.grad_y : &a.y, backward ? &a.grad_x : &a.y,
                        backward ? &a.grad_z : &a.y};
  bool pieces = a.D % V == 0;
  for (const Tok* t : used)
    pieces = pieces && (t->p == nullptr ||
                        (t->sb % V == 0 && t->sl % V == 0 && t->sh % V == 0 &&
                         reinterpret_cast<uintptr_t>(t->p) % 16 == 0));
  return a.z.p ? norm_by_size<Act, true>(a, backward, pieces, st)
               : norm_by_size<Act, false>(a, backward, pieces, st);
}

}  // namespace gdnq
