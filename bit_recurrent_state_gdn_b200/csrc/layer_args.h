// Kernel arguments and launch interface of the operators around the recurrence (gdnq_layer.h).
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

#include "gdnq_layer.h"

namespace gdnq {

// A token array on the device: element (b, l, h, d) at p[b sb + l sl + h sh + d].
struct Tok {
  void* p;
  int64_t sb, sl, sh;
};

struct ScanArgs {
  Tok x, g, o;            // forward; the backward pass reads x and g
  Tok grad_o, grad_x, grad_g;
  const float* h0;        // forward: h0; backward: grad_hT
  float* hT;              // forward: hT; backward: grad_h0
  float* hist;            // written forward, read backward
  const int32_t* lens;
  int B, L, H, D, C;      // C = H D
  void* spans;            // workspace: what each span of a split sequence does to the state
  int span_tokens;        // tokens of a span; spans per sequence
  int spans_per_unit;
};

struct NormArgs {
  Tok x, z, y;
  Tok grad_y, grad_x, grad_z;
  const float* w;
  const float* bias;
  float* grad_w;
  float* grad_bias;
  float* partials;        // backward: workspace
  const int32_t* lens;
  float eps, inv_d;
  int B, L, H, D;
  int center, activation, per_channel;
};

struct ConvArgs {
  Tok x, y;
  Tok grad_y, grad_x;
  const float* w;
  const float* bias;
  const void* state_in;
  void* state_out;
  const void* grad_state_out;
  void* grad_state_in;
  float* grad_w;
  float* grad_bias;
  float* partials;
  const int32_t* lens;
  int B, L, H, D, C, K;
  int activation;
};

// The SMs that work is shared out over: a constant, since the sizes of workspaces follow from it and
// are answered on the host, whatever device is current then.
constexpr int kSms = 148;

// Into how many parts each of `units` equal pieces of work goes on a machine that holds `slots`
// parts at a time: as many as fit at once, or where fewer than four of them do (so that rounding
// down would leave much of the machine idle) enough for four turns.
inline int64_t shares(int64_t slots, int64_t units) {
  const int64_t fit = slots / units;
  return fit >= 4 ? fit : (4 * slots + units - 1) / units;
}

// Launches the kernel that adds partial sums behind the one that forms them, so that its launch
// overlaps that one's end (the kernels say let_next_launch and wait_for_last).
template <typename... Params>
cudaError_t launch_behind(void (*kernel)(Params...), unsigned grid, int threads, cudaStream_t st,
                          Params... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Forward or backward scan, by activation type; scale is a gdn_input_scale.
cudaError_t launch_scan_f32(const ScanArgs& a, int scale, bool backward, cudaStream_t st);
cudaError_t launch_scan_bf16(const ScanArgs& a, int scale, bool backward, cudaStream_t st);
// Fills in span_tokens and spans_per_unit, and returns the bytes of `spans` (0: not split).
size_t scan_spans(ScanArgs& a);
cudaError_t launch_norm_f32_forward(const NormArgs& a, cudaStream_t st);
cudaError_t launch_norm_f32_backward(const NormArgs& a, cudaStream_t st);
cudaError_t launch_norm_bf16_forward(const NormArgs& a, cudaStream_t st);
cudaError_t launch_norm_bf16_backward(const NormArgs& a, cudaStream_t st);
size_t norm_backward_workspace(const gdn_norm_config& cfg, int L);
cudaError_t launch_conv_f32(const ConvArgs& a, bool backward, cudaStream_t st);
cudaError_t launch_conv_bf16(const ConvArgs& a, bool backward, cudaStream_t st);
size_t conv_backward_workspace(const gdn_conv_config& cfg, int L);

}  // namespace gdnq
