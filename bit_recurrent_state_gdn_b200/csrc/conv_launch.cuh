// Launches of the short-convolution kernels for one activation type.
#pragma once

#include <algorithm>

#include "conv_kernels.cuh"
#include "window_dispatch.cuh"

#ifndef CF
#define CF 2
#define VF 16
#define CSF 3
#define CWAVE 1
#define CDEC 1
#endif
#ifndef CB
#define CB 2
#define CSB 3
#define CBK 1
#endif
namespace gdnq {

// Tokens of a run at least: the K - 1 tokens before it are read twice.
constexpr int kConvRun = 16;

inline ConvSplit conv_runs(int B, int L, int columns, int64_t threads) {
  ConvSplit s;
  s.columns = columns;
  const int64_t want = std::max<int64_t>(1, threads / std::max<int64_t>(1, (int64_t)B * columns));
  const int64_t most = std::max<int64_t>(1, L / kConvRun);
  const int64_t runs = std::min(want, most);
  s.run_tokens = (int)std::max<int64_t>(1, (L + runs - 1) / runs);
  s.runs = (int)std::max<int64_t>(1, ((int64_t)L + s.run_tokens - 1) / s.run_tokens);
  s.parts = 1;
  return s;
}

inline ConvSplit conv_forward_split(int B, int L, int columns) {
  const int64_t threads = (int64_t)148 * CF * kConvThreads * (L < 8 ? CDEC : CWAVE);
  ConvSplit s = conv_runs(B, L, columns, threads);
  s.parts = (int)std::min<int64_t>((int64_t)B * s.runs, std::max<int64_t>(1, threads / columns));
  return s;
}

inline ConvSplit conv_backward_split(int B, int L, int C, int V) {
  const int columns = (C + V - 1) / V, slabs = (columns + 31) / 32;
  const int64_t parts = std::max(1, 148 * CB / slabs), rows = parts * (kConvThreads / 32);
  ConvSplit s = conv_runs(B, L, columns, rows * columns * CBK);
  s.parts = (int)std::min<int64_t>(parts, ((int64_t)B * s.runs + kConvThreads / 32 - 1) / (kConvThreads / 32));
  return s;
}

cudaError_t launch_conv_reduce(const ConvArgs& a, int parts, cudaStream_t st);

template <typename Act, int K, bool SILU, class F, class B>
cudaError_t conv_go(const ConvArgs& a, bool backward, cudaStream_t st) {
  if (!backward) {
    constexpr auto kernel = conv_kernel<Act, K, SILU, F, CF>;
    const cudaError_t e = ensure_smem<kernel>(F::kBytes);
    if (e != cudaSuccess) return e;
    const ConvSplit s = conv_forward_split(a.B, a.L, (a.C + F::V - 1) / F::V);
    const int64_t threads = (int64_t)s.parts * s.columns;
    kernel<<<(unsigned)((threads + kConvThreads - 1) / kConvThreads), kConvThreads, F::kBytes, st>>>(a, s);
    return cudaGetLastError();
  }
  constexpr auto kernel = conv_backward_kernel<Act, K, SILU, B, 32, CB>;
  constexpr int kShared = conv_backward_shared<K, 32, B>();
  cudaError_t e = ensure_smem<kernel>(kShared);
  if (e != cudaSuccess) return e;
  const ConvSplit s = conv_backward_split(a.B, a.L, a.C, B::V);
  const int slabs = (s.columns + 31) / 32;
  kernel<<<(unsigned)slabs * (unsigned)s.parts, kConvThreads, kShared, st>>>(a, s);
  e = cudaGetLastError();
  return e == cudaSuccess ? launch_conv_reduce(a, s.parts, st) : e;
}

template <typename Act, int K, bool SILU>
cudaError_t conv_by_place(const ConvArgs& a, bool backward, bool pieces, cudaStream_t st) {
  if (pieces)
    return conv_go<Act, K, SILU, RowsInShared<Act, VF / (int)sizeof(Act), K, 1, CSF>,
                   RowsInShared<Act, 4, K, 2, CSB>>(a, backward, st);
  return conv_go<Act, K, SILU, RowsInRegisters<Act, K, 1>, RowsInRegisters<Act, K, 2>>(a, backward, st);
}

template <typename Act, int K>
cudaError_t conv_by_act(const ConvArgs& a, bool backward, bool pieces, cudaStream_t st) {
  return a.activation == GDN_ACT_SILU ? conv_by_place<Act, K, true>(a, backward, pieces, st)
                                      : conv_by_place<Act, K, false>(a, backward, pieces, st);
}

template <typename Act>
cudaError_t launch_conv_as(ConvArgs a, bool backward, cudaStream_t st) {
  const Tok* used[3] = {&a.x, backward ? &a.grad_y : &a.y, backward ? &a.grad_x : &a.y};
  const void* states[4] = {a.state_in, a.state_out, a.grad_state_in, a.grad_state_out};
  // where a token's heads follow one another in every array, they are one head of C channels
  bool dense = true;
  for (const Tok* t : used) dense = dense && t->sh == a.D;
  if (dense || a.H == 1) {
    a.D = a.C;
    a.H = 1;
    a.x.sh = a.y.sh = a.grad_y.sh = a.grad_x.sh = 0;
  }
  // vectors of V channels in one head, aligned: 16 bytes, backward those of 4 channels
  const int V = backward ? 4 : VF / (int)sizeof(Act);
  bool pieces = a.L > 0 && a.D % V == 0;
  for (const Tok* t : used)
    pieces = pieces && t->sb % V == 0 && t->sl % V == 0 && t->sh % V == 0 &&
             reinterpret_cast<uintptr_t>(t->p) % (V * sizeof(Act)) == 0;
  for (const void* s : states) pieces = pieces && reinterpret_cast<uintptr_t>(s) % (V * sizeof(Act)) == 0;
  switch (a.K) {
    case 2:
      return conv_by_act<Act, 2>(a, backward, pieces, st);
    case 3:
      return conv_by_act<Act, 3>(a, backward, pieces, st);
    default:
      return conv_by_act<Act, 4>(a, backward, pieces, st);
  }
}

}  // namespace gdnq
