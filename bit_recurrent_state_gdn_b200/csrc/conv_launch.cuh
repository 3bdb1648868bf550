// Launches of the short-convolution kernels for one activation type.
#pragma once

#include <algorithm>

#include "conv_kernels.cuh"
#include "window_dispatch.cuh"

namespace gdnq {

// CTAs per SM that the kernels' registers are bounded for. Three of the run kernels spill (8 x 4096
// channels x 4096 tokens forward 107 us against 96; backward 4 sequences 220 against 95).
constexpr int kConvResident = 2, kConvStepResident = 4;
// Channels of a thread backward (with 2: 125 us against 95), and for one token, whose K rows of
// several sequences are in registers (8 channels: 18.4 us against 16.3, 1024 x 4096 channels).
constexpr int kConvBackVec = 4, kConvStepVec = 4;

// Tokens of a run at least: the K - 1 tokens before it (backward, also behind it) are read twice. It
// counts where sequences are short or few, bf16, forward / backward, with 16 / 32 / 64: 512 channels x
// 1024 tokens 8.6 / 12.5 / 18.7 us and 12.4 / 15.6 / 20.8; 2 x 1024 channels x 16384 29 / 29 / 31 and
// 50 / 50 / 50; more work than that is shared out by slots.
constexpr int kConvRun = 32;

inline ConvSplit conv_split(int B, int L, int columns, int64_t threads) {
  ConvSplit s;
  s.columns = columns;
  const int64_t runs = std::min(shares(threads, std::max<int64_t>(1, (int64_t)B * columns)),
                                std::max<int64_t>(1, L / kConvRun));
  s.run_tokens = (int)std::max<int64_t>(1, (L + runs - 1) / runs);
  s.runs = (int)std::max<int64_t>(1, ((int64_t)L + s.run_tokens - 1) / s.run_tokens);
  s.parts = (int)std::min<int64_t>((int64_t)B * s.runs, std::max<int64_t>(1, threads / columns));
  return s;
}

// Columns of a backward CTA: a warp's, or eight where there are not many (73 x 32 channels x 15613
// tokens: 163 us with 24 of 32 lanes idle).
inline int conv_back_columns(int columns) { return columns <= 16 ? 8 : 32; }

inline ConvSplit conv_backward_split(int B, int L, int C, int V) {
  const int columns = (C + V - 1) / V, wide = conv_back_columns(columns);
  const int slabs = (columns + wide - 1) / wide, kRows = kConvThreads / wide;
  const int64_t parts = std::max(1, kSms * kConvResident / slabs);
  ConvSplit s = conv_split(B, L, columns, parts * kRows * columns);
  s.parts = (int)std::min<int64_t>(parts, ((int64_t)B * s.runs + kRows - 1) / kRows);
  return s;
}

cudaError_t launch_conv_reduce(const ConvArgs& a, int parts, cudaStream_t st);

template <typename Act, int K, bool SILU, class Rows, int TX>
cudaError_t conv_back(const ConvArgs& a, const ConvSplit& s, cudaStream_t st) {
  constexpr auto kernel = conv_backward_kernel<Act, K, SILU, Rows, TX, kConvResident>;
  constexpr int kShared = conv_backward_shared<K, TX, Rows>();
  cudaError_t e = ensure_smem<kernel>(kShared);
  if (e != cudaSuccess) return e;
  const int slabs = (s.columns + TX - 1) / TX;
  kernel<<<(unsigned)slabs * (unsigned)s.parts, kConvThreads, kShared, st>>>(a, s);
  e = cudaGetLastError();
  return e == cudaSuccess ? launch_conv_reduce(a, s.parts, st) : e;
}

template <int N>
struct StepVec {
  static constexpr int V = N;
};

template <typename Act, int K, bool SILU, class F, class B, class S>
cudaError_t conv_go(const ConvArgs& a, bool backward, cudaStream_t st) {
  if (!backward && a.L == 1) {
    // a thread takes several sequences where there are more than fill the machine
    const ConvSplit s = conv_split(a.B, 1, (a.C + S::V - 1) / S::V,
                                   (int64_t)kSms * kConvStepResident * kConvThreads);
    const int64_t threads = (int64_t)s.parts * s.columns;
    const unsigned grid = (unsigned)((threads + kConvThreads - 1) / kConvThreads);
    if (s.parts == a.B)
      conv_step_kernel<Act, K, SILU, S::V, 1, kConvStepResident><<<grid, kConvThreads, 0, st>>>(a, s);
    else
      conv_step_kernel<Act, K, SILU, S::V, 2, kConvStepResident><<<grid, kConvThreads, 0, st>>>(a, s);
    return cudaGetLastError();
  }
  if (!backward) {
    // single channels have fewer registers to keep, and fewer bytes in flight each: four (162 x 29
    // channels, 3 x 12237 tokens: 1.9 TB/s against 1.3 with two)
    constexpr int kResident = F::V == 1 ? 4 : kConvResident;
    constexpr auto kernel = conv_kernel<Act, K, SILU, F, kResident>;
    const cudaError_t e = ensure_smem<kernel>(F::kBytes);
    if (e != cudaSuccess) return e;
    const ConvSplit s = conv_split(a.B, a.L, (a.C + F::V - 1) / F::V,
                                   (int64_t)kSms * kResident * kConvThreads);
    const int64_t threads = (int64_t)s.parts * s.columns;
    kernel<<<(unsigned)((threads + kConvThreads - 1) / kConvThreads), kConvThreads, F::kBytes, st>>>(a, s);
    return cudaGetLastError();
  }
  const ConvSplit s = conv_backward_split(a.B, a.L, a.C, B::V);
  return conv_back_columns(s.columns) == 8 ? conv_back<Act, K, SILU, B, 8>(a, s, st)
                                           : conv_back<Act, K, SILU, B, 32>(a, s, st);
}

template <typename Act, int K, bool SILU>
cudaError_t conv_by_place(const ConvArgs& a, bool backward, int wide, cudaStream_t st) {
  constexpr int V = 16 / (int)sizeof(Act);
  if (wide >= (backward ? kConvBackVec : V))
    return conv_go<Act, K, SILU, RowsInShared<Act, V, K, 1, 3>, RowsInShared<Act, kConvBackVec, K, 2, 3>,
                   StepVec<kConvStepVec>>(a, backward, st);
  if (wide >= 2)
    return conv_go<Act, K, SILU, RowsInShared<Act, 2, K, 1, 4>, RowsInShared<Act, 2, K, 2, 3>,
                   StepVec<2>>(a, backward, st);
  return conv_go<Act, K, SILU, RowsInRegisters<Act, K, 1>, RowsInRegisters<Act, K, 2>, StepVec<1>>(
      a, backward, st);
}

template <typename Act, int K>
cudaError_t conv_by_act(const ConvArgs& a, bool backward, int wide, cudaStream_t st) {
  return a.activation == GDN_ACT_SILU ? conv_by_place<Act, K, true>(a, backward, wide, st)
                                      : conv_by_place<Act, K, false>(a, backward, wide, st);
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
  // the most channels that lie in one head and are aligned wherever they begin
  int wide = a.L > 0 ? 16 / (int)sizeof(Act) : 1;
  for (bool fits = false; !fits && wide > 1; wide /= fits ? 1 : 2) {
    fits = a.D % wide == 0;
    for (const Tok* t : used)
      fits = fits && t->sb % wide == 0 && t->sl % wide == 0 && t->sh % wide == 0 &&
             reinterpret_cast<uintptr_t>(t->p) % (wide * sizeof(Act)) == 0;
    for (const void* s : states) fits = fits && reinterpret_cast<uintptr_t>(s) % (wide * sizeof(Act)) == 0;
  }
  switch (a.K) {
    case 2:
      return conv_by_act<Act, 2>(a, backward, wide, st);
    case 3:
      return conv_by_act<Act, 3>(a, backward, wide, st);
    default:
      return conv_by_act<Act, 4>(a, backward, wide, st);
  }
}

}  // namespace gdnq
