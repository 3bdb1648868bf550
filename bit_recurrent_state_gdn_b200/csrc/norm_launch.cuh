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

// Channels of a head that a warp may hold. 4 x 4096 tokens, gated bf16 rows, forward / backward: 12
// rows of 640 a token 212 / 432 us (a CTA a row: 578 / 828), 8 rows of 1024 135 / 312 (419 / 564), in
// fp32 255 / 485 (394 / 545). Only few rows are served sooner by a CTA each: 512 of 1024 channels
// 14.3 / 20.2 (8.0 / 12.3).
constexpr int kNormWarp = 1024;

// CTAs of the kernels for rows of more channels: eight an SM. 32768 gated bf16 rows, with 4 / 8 / 16 an
// SM: of 2048 channels forward 190 / 182 / 158 us, backward 326 / 269 / 272; of 4096 304 / 300 / 296 and
// 820 / 826 / 849. 4096 fp32 rows of 4096, whose partial sums count, backward 96 / 107 / 130.
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
  return backward ? (channels <= 8 ? 2 : 1) : (channels <= 8 ? 3 : channels <= 16 ? 2 : 1);
}

template <typename Act, bool GATE, bool BACKWARD, class P>
cudaError_t norm_go(const NormArgs& a, cudaStream_t st) {
  constexpr int kResident = norm_resident(P::NI * P::V, BACKWARD);
  const NormSplit s = norm_plan(a.D, a.H, (int64_t)a.B * a.L, sizeof(Act), P::LANES, kResident);
  const unsigned grid = (unsigned)s.parts * (unsigned)s.heads_of_blocks;
  if constexpr (!BACKWARD) {
    constexpr auto kernel = norm_kernel<Act, GATE, P, kResident>;
    const cudaError_t e = ensure_smem<kernel>(P::kBytes);
    if (e != cudaSuccess) return e;
    kernel<<<grid, kNormThreads, P::kBytes, st>>>(a, s);
    return cudaGetLastError();
  } else {
    constexpr auto kernel = norm_backward_kernel<Act, GATE, P, kResident>;
    constexpr int kShared = norm_backward_shared<P>();
    cudaError_t e = ensure_smem<kernel>(kShared);
    if (e != cudaSuccess) return e;
    kernel<<<grid, kNormThreads, kShared, st>>>(a, s);
    e = cudaGetLastError();
    return e == cudaSuccess ? launch_norm_reduce(a, norm_partials(s, a.H, a.per_channel), st) : e;
  }
}

// Rows of the ring by the bytes of each array that a lane holds of a row. Half as many / these / half as
// many again, 32768 tokens of 4096 channels, gated bf16: rows of 32 (16 bytes) forward 153 / 134 / 148
// us, backward 257 / 224 / 243; of 128 153 / 138 / 138 and 256 / 243 / 240; of 512 (32 bytes)
// 134 / 146 / 153 and 255 / 238 / 244; of 1024 (64 bytes) 139 / 136 / 131 and 308 / 306 / 318.
constexpr int norm_stages(int bytes, bool backward) {
  return bytes <= 4 ? 8 : bytes <= 8 ? 6 : bytes <= 16 ? 4 : bytes <= 32 ? (backward ? 3 : 4)
                    : bytes <= 64 ? (backward ? 2 : 3) : 2;
}

// Pieces of V channels (V = 0: single ones that no asynchronous copy can take).
template <typename Act, bool GATE, bool BACKWARD, int V, int LANES, int NI>
cudaError_t norm_pieces(const NormArgs& a, cudaStream_t st) {
  constexpr int N = (GATE ? 2 : 1) + (BACKWARD ? 1 : 0);
  if constexpr (V == 0)
    return norm_go<Act, GATE, BACKWARD, PiecesInRegisters<Act, LANES, NI, N>>(a, st);
  else
    return norm_go<Act, GATE, BACKWARD,
                   PiecesInShared<Act, V, LANES, NI, N, norm_stages(NI * V * (int)sizeof(Act), BACKWARD),
                                  !BACKWARD>>(a, st);
}

template <typename Act, bool BACKWARD, int NI>
cudaError_t norm_wide(const NormArgs& a, cudaStream_t st) {
  const int64_t tokens = (int64_t)a.B * a.L;
  if constexpr (!BACKWARD) {
    norm_wide_kernel<Act, NI><<<(unsigned)std::min<int64_t>(tokens * a.H, kSms * 8), kNormThreads, 0, st>>>(a);
    return cudaGetLastError();
  } else {
    const int parts = norm_wide_parts(tokens, a.H);
    norm_wide_backward_kernel<Act, NI><<<(unsigned)parts * (unsigned)a.H, kNormThreads, 0, st>>>(a, parts);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? launch_norm_reduce(a, (int64_t)parts * a.H, st) : e;
  }
}

// Lanes and pieces per lane for rows of n pieces; cudaErrorNotSupported where a warp does not hold
// them. A row costs a lane much the same however few channels it has there, so that a lane takes
// 16 bytes of each array at the least (4 x 55 x 4096 rows of 36 channels backward, one piece of 8
// bytes a lane: 2.2 TB/s).
template <typename Act, bool GATE, bool BACKWARD, int V>
cudaError_t norm_by_pieces(const NormArgs& a, int n, cudaStream_t st) {
  constexpr int F = V == 0 ? 4 : 16 / (V * (int)sizeof(Act));
  if (n <= 2 * F) return norm_pieces<Act, GATE, BACKWARD, V, 2, F>(a, st);
  if (n <= 4 * F) return norm_pieces<Act, GATE, BACKWARD, V, 4, F>(a, st);
  if (n <= 8 * F) return norm_pieces<Act, GATE, BACKWARD, V, 8, F>(a, st);
  if (n <= 16 * F) return norm_pieces<Act, GATE, BACKWARD, V, 16, F>(a, st);
  if (n <= 32 * F) return norm_pieces<Act, GATE, BACKWARD, V, 32, F>(a, st);
  if (n <= 64 * F) return norm_pieces<Act, GATE, BACKWARD, V, 32, 2 * F>(a, st);
  if (n <= 128 * F) return norm_pieces<Act, GATE, BACKWARD, V, 32, 4 * F>(a, st);
  if constexpr (V * sizeof(Act) == 16 && sizeof(Act) == 4)
    if (n <= 256) return norm_pieces<Act, GATE, BACKWARD, V, 32, 8>(a, st);
  return cudaErrorNotSupported;
}

// `wide`: channels that may be moved as one.
template <typename Act, bool GATE, bool BACKWARD>
cudaError_t norm_by_place(const NormArgs& a, int wide, cudaStream_t st) {
  constexpr int V = 16 / (int)sizeof(Act);
  cudaError_t e = cudaErrorNotSupported;
  if (a.D <= kNormWarp) {
    if (wide == V)
      e = norm_by_pieces<Act, GATE, BACKWARD, V>(a, a.D / V, st);
    else if (wide == V / 2)
      e = norm_by_pieces<Act, GATE, BACKWARD, V / 2>(a, a.D / (V / 2), st);
    else if (wide == V / 4)
      e = norm_by_pieces<Act, GATE, BACKWARD, V / 4>(a, a.D / (V / 4), st);
    else if constexpr (V == 8)  // single bf16 elements
      e = norm_by_pieces<Act, GATE, BACKWARD, 0>(a, a.D, st);
  }
  if (e != cudaErrorNotSupported) return e;
  if (a.D <= 1024) return norm_wide<Act, BACKWARD, 4>(a, st);
  if (a.D <= 2048) return norm_wide<Act, BACKWARD, 8>(a, st);
  if (a.D <= 4096) return norm_wide<Act, BACKWARD, 16>(a, st);
  return norm_wide<Act, BACKWARD, 32>(a, st);
}

template <typename Act, bool BACKWARD>
cudaError_t launch_norm_as(const NormArgs& a, cudaStream_t st) {
  const Tok* used[5] = {&a.x, &a.z, BACKWARD ? &a.grad_y : &a.y, BACKWARD ? &a.grad_x : &a.y,
                        BACKWARD ? &a.grad_z : &a.y};
  int wide = 16 / (int)sizeof(Act);
  for (bool fits = false; !fits && wide > 1; wide /= fits ? 1 : 2) {
    fits = a.D % wide == 0;
    for (const Tok* t : used)
      fits = fits && (t->p == nullptr ||
                      (t->sb % wide == 0 && t->sl % wide == 0 && t->sh % wide == 0 &&
                       reinterpret_cast<uintptr_t>(t->p) % (wide * sizeof(Act)) == 0));
  }
  return a.z.p ? norm_by_place<Act, true, BACKWARD>(a, wide, st)
               : norm_by_place<Act, false, BACKWARD>(a, wide, st);
}

}  // namespace gdnq
