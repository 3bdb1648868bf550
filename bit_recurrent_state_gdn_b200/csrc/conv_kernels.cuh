// Causal depthwise convolution over a few tokens, with SiLU, and its gradients
// (include/gdnq_layer.h). One thread walks a run of tokens of one channel, the last K inputs in
// registers.
#pragma once

#include "layer_util.cuh"

namespace gdnq {

constexpr int kConvRun = 32;  // tokens per thread and run

// Input of token t of channel c: x, or the state before the first token.
template <typename Act, int K>
__device__ __forceinline__ float conv_input(const ConvArgs& a, const Act* x, int b, int c, int t) {
  if (t >= 0) return Num<Act>::to_f(x[t * a.x.sl]);
  const Act* s = static_cast<const Act*>(a.state_in);
  return s ? Num<Act>::to_f(s[((int64_t)b * (K - 1) + t + K - 1) * a.C + c]) : 0.0f;
}

template <typename Act, int K>
__global__ void __launch_bounds__(256) conv_kernel(ConvArgs a, int runs) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int c = (int)(i % a.C);
  const int64_t r = i / a.C;
  if (r >= (int64_t)a.B * runs) return;
  const int b = (int)(r / runs), t0 = (int)(r % runs) * kConvRun;
  const int len = seq_len(a.lens, b, a.L), t1 = min(t0 + kConvRun, len);
  if (t0 > 0 && t0 >= len) return;
  const int hd = c / a.D, d = c % a.D;
  const Act* x = static_cast<const Act*>(a.x.p) + channel_offset(a.x, b, hd, d);
  Act* y = static_cast<Act*>(a.y.p) + channel_offset(a.y, b, hd, d);
  float w[K], v[K];
#pragma unroll
  for (int j = 0; j < K; ++j) w[j] = a.w[(int64_t)c * K + j];
  const float bias = a.bias ? a.bias[c] : 0.0f;
#pragma unroll
  for (int j = 0; j < K - 1; ++j) v[j + 1] = conv_input<Act, K>(a, x, b, c, t0 - K + 1 + j);
  // the run that begins the sequence also hands the state on: it alone reads state_in, so
  // state_out may be the same array
  if (t0 == 0 && a.state_out) {
    float s[K - 1];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) s[j] = conv_input<Act, K>(a, x, b, c, len - K + 1 + j);
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
      static_cast<Act*>(a.state_out)[((int64_t)b * (K - 1) + j) * a.C + c] = Num<Act>::from_f(s[j]);
  }
  for (int t = t0; t < t1; ++t) {
#pragma unroll
    for (int j = 0; j < K - 1; ++j) v[j] = v[j + 1];
    v[K - 1] = Num<Act>::to_f(x[t * a.x.sl]);
    float p = bias;
#pragma unroll
    for (int j = 0; j < K; ++j) p = fmaf(w[j], v[j], p);
    y[t * a.y.sl] = Num<Act>::from_f(a.activation == GDN_ACT_SILU ? p * sigmoidf(p) : p);
  }
}

// CTA = 32 channels x 8 runs at a time; its sums of dp x and dp go to partials[part][C][K + 1].
template <typename Act, int K>
__global__ void __launch_bounds__(256) conv_backward_kernel(ConvArgs a, int runs, int slabs) {
  __shared__ float sum[8][32][K + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int slab = blockIdx.x % slabs, part = blockIdx.x / slabs, parts = gridDim.x / slabs;
  const int c = slab * 32 + lane;
  float w[K], dw[K], db = 0.0f, bias = 0.0f;
#pragma unroll
  for (int j = 0; j < K; ++j) dw[j] = 0.0f;
  if (c < a.C) {
    const int hd = c / a.D, d = c % a.D;
#pragma unroll
    for (int j = 0; j < K; ++j) w[j] = a.w[(int64_t)c * K + j];
    if (a.bias) bias = a.bias[c];
    const Act* gso = static_cast<const Act*>(a.grad_state_out);
    Act* gsi = static_cast<Act*>(a.grad_state_in);
    for (int64_t r = (int64_t)part * 8 + warp; r < (int64_t)a.B * runs; r += (int64_t)parts * 8) {
      const int b = (int)(r / runs), t0 = (int)(r % runs) * kConvRun;
      const int len = seq_len(a.lens, b, a.L), t1 = min(t0 + kConvRun, len);
      if (t0 > 0 && t0 >= len) continue;
      const Act* x = static_cast<const Act*>(a.x.p) + channel_offset(a.x, b, hd, d);
      const Act* gy = static_cast<const Act*>(a.grad_y.p) + channel_offset(a.grad_y, b, hd, d);
      Act* gx = static_cast<Act*>(a.grad_x.p) + channel_offset(a.grad_x, b, hd, d);
      float v[K], dp[K];  // inputs t-K+1 .. t; dp[j] of token t - j
#pragma unroll
      for (int j = 0; j < K; ++j) dp[j] = 0.0f;
#pragma unroll
      for (int j = 0; j < K - 1; ++j) v[j + 1] = conv_input<Act, K>(a, x, b, c, t0 - K + 1 + j);
      for (int t = t0; t < t1 + K - 1; ++t) {
#pragma unroll
        for (int j = K - 1; j > 0; --j) dp[j] = dp[j - 1];
        dp[0] = 0.0f;
        if (t < len) {
#pragma unroll
          for (int j = 0; j < K - 1; ++j) v[j] = v[j + 1];
          v[K - 1] = Num<Act>::to_f(x[t * a.x.sl]);
          float p = bias;
#pragma unroll
          for (int j = 0; j < K; ++j) p = fmaf(w[j], v[j], p);
          dp[0] = Num<Act>::to_f(gy[t * a.grad_y.sl]);
          if (a.activation == GDN_ACT_SILU) {
            const float q = sigmoidf(p);
            dp[0] *= q * fmaf(p, 1.0f - q, 1.0f);
          }
          if (t < t1) {
            db += dp[0];
#pragma unroll
            for (int j = 0; j < K; ++j) dw[j] = fmaf(dp[0], v[j], dw[j]);
          }
        }
        // the gradient of input s = t - K + 1 is complete
        const int s = t - (K - 1), u = t - len;
        if (s < t0 && t0 > 0) continue;
        float g = 0.0f;
#pragma unroll
        for (int j = 0; j < K; ++j) g = fmaf(w[j], dp[j], g);
        if (gso && u >= 0) g += Num<Act>::to_f(gso[((int64_t)b * (K - 1) + u) * a.C + c]);
        if (s >= 0)
          gx[s * a.grad_x.sl] = Num<Act>::from_f(g);
        else if (gsi)
          gsi[((int64_t)b * (K - 1) + t) * a.C + c] = Num<Act>::from_f(g);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < K; ++j) sum[warp][lane][j] = dw[j];
  sum[warp][lane][K] = db;
  __syncthreads();
  if (warp == 0 && c < a.C) {
    float* p = a.partials + ((int64_t)part * a.C + c) * (K + 1);
#pragma unroll
    for (int j = 0; j <= K; ++j) {
      float s = 0.0f;
      for (int q = 0; q < 8; ++q) s += sum[q][lane][j];
      p[j] = s;
    }
  }
}

// grad_w and grad_bias: the sum over the parts, in order.
template <int K>
__global__ void __launch_bounds__(128) conv_reduce_kernel(ConvArgs a, int parts) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, n = (int64_t)a.C * (K + 1);
  if (i >= n) return;
  float s = 0.0f;
  for (int p = 0; p < parts; ++p) s += a.partials[p * n + i];
  const int64_t c = i / (K + 1);
  const int j = (int)(i % (K + 1));
  if (j < K)
    a.grad_w[c * K + j] = s;
  else if (a.grad_bias)
    a.grad_bias[c] = s;
}

}  // namespace gdnq
