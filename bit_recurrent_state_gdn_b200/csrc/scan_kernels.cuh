// Gated scan h_t = a_t h_{t-1} + s(g_t) x_t, a_t = e^{g_t}, and its gradients
// (include/gdnq_layer.h). One thread per (sequence, channel) walks the tokens.
#pragma once

#include "layer_util.cuh"

namespace gdnq {

// s(g) and s'(g).
template <int SCALE>
__device__ __forceinline__ float scan_factor(float g) {
  if constexpr (SCALE == GDN_SCALE_COMPLEMENT) return -expm1f(g);
  if constexpr (SCALE == GDN_SCALE_SQRT) return sqrtf(-expm1f(2.0f * g));
  return 1.0f;
}

template <int SCALE>
__device__ __forceinline__ float scan_factor_slope(float a, float s) {
  if constexpr (SCALE == GDN_SCALE_COMPLEMENT) return -a;
  if constexpr (SCALE == GDN_SCALE_SQRT) return s > 0.0f ? -a * a / s : 0.0f;
  return 0.0f;
}

template <typename Act, int SCALE>
__global__ void __launch_bounds__(128) scan_kernel(ScanArgs a) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= (int64_t)a.B * a.C) return;
  const int b = (int)(i / a.C), c = (int)(i % a.C), hd = c / a.D, d = c % a.D;
  const int len = seq_len(a.lens, b, a.L);
  const Act* x = static_cast<const Act*>(a.x.p) + channel_offset(a.x, b, hd, d);
  const float* g = static_cast<const float*>(a.g.p) + channel_offset(a.g, b, hd, d);
  Act* o = static_cast<Act*>(a.o.p) + channel_offset(a.o, b, hd, d);
  const int64_t nchunk = (a.L + GDN_SCAN_CHUNK - 1) / GDN_SCAN_CHUNK;
  float h = a.h0 ? a.h0[i] : 0.0f;
  for (int t = 0; t < len; ++t) {
    if (a.hist && t % GDN_SCAN_CHUNK == 0)
      a.hist[(b * nchunk + t / GDN_SCAN_CHUNK) * a.C + c] = h;
    const float gt = g[t * a.g.sl];
    h = fmaf(expf(gt), h, scan_factor<SCALE>(gt) * Num<Act>::to_f(x[t * a.x.sl]));
    o[t * a.o.sl] = Num<Act>::from_f(h);
  }
  if (a.hT) a.hT[i] = h;
}

template <typename Act, int SCALE>
__global__ void __launch_bounds__(128) scan_backward_kernel(ScanArgs a) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= (int64_t)a.B * a.C) return;
  const int b = (int)(i / a.C), c = (int)(i % a.C), hd = c / a.D, d = c % a.D;
  const int len = seq_len(a.lens, b, a.L);
  const Act* x = static_cast<const Act*>(a.x.p) + channel_offset(a.x, b, hd, d);
  const float* g = static_cast<const float*>(a.g.p) + channel_offset(a.g, b, hd, d);
  const Act* go = static_cast<const Act*>(a.grad_o.p) + channel_offset(a.grad_o, b, hd, d);
  Act* gx = static_cast<Act*>(a.grad_x.p) + channel_offset(a.grad_x, b, hd, d);
  float* gg = static_cast<float*>(a.grad_g.p) + channel_offset(a.grad_g, b, hd, d);
  const int64_t nchunk = (a.L + GDN_SCAN_CHUNK - 1) / GDN_SCAN_CHUNK;
  float carry = a.h0 ? a.h0[i] : 0.0f;  // a_{t+1} dh_{t+1}
  for (int t0 = (len - 1) / GDN_SCAN_CHUNK * GDN_SCAN_CHUNK; len > 0 && t0 >= 0;
       t0 -= GDN_SCAN_CHUNK) {
    const int n = min(GDN_SCAN_CHUNK, len - t0);
    float prev[GDN_SCAN_CHUNK];  // the state before each token
    float h = a.hist[(b * nchunk + t0 / GDN_SCAN_CHUNK) * a.C + c];
    for (int j = 0; j < n; ++j) {
      const float gt = g[(t0 + j) * a.g.sl];
      prev[j] = h;
      h = fmaf(expf(gt), h, scan_factor<SCALE>(gt) * Num<Act>::to_f(x[(t0 + j) * a.x.sl]));
    }
    for (int j = n - 1; j >= 0; --j) {
      const int64_t t = t0 + j;
      const float gt = g[t * a.g.sl], at = expf(gt), s = scan_factor<SCALE>(gt);
      const float dh = Num<Act>::to_f(go[t * a.grad_o.sl]) + carry;
      gx[t * a.grad_x.sl] = Num<Act>::from_f(s * dh);
      carry = at * dh;
      gg[t * a.grad_g.sl] = fmaf(
          carry, prev[j], scan_factor_slope<SCALE>(at, s) * Num<Act>::to_f(x[t * a.x.sl]) * dh);
    }
  }
  if (a.hT) a.hT[i] = carry;
}

}  // namespace gdnq
