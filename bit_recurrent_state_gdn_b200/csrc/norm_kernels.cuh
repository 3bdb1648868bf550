// Group norm over each head's channels with an activation or a gate, and its gradients
// (include/gdnq_layer.h). One CTA of 256 threads takes a (token, head) row at a time, NI channels
// per thread in registers.
#pragma once

#include "layer_util.cuh"

namespace gdnq {

constexpr int kNormThreads = 256;

// act(u) and act'(u).
__device__ __forceinline__ float2 act_slope(int activation, float u) {
  if (activation == GDN_ACT_NONE) return make_float2(u, 1.0f);
  const float q = sigmoidf(u);
  if (activation == GDN_ACT_SIGMOID) return make_float2(q, q * (1.0f - q));
  return make_float2(u * q, q * fmaf(u, 1.0f - q, 1.0f));
}

// Sums of (p, q) over the CTA, the same in every thread.
__device__ __forceinline__ float2 cta_sum(float p, float q) {
  __shared__ float2 part[kNormThreads / 32];
#pragma unroll
  for (int m = 16; m; m >>= 1) {
    p += __shfl_xor_sync(~0u, p, m);
    q += __shfl_xor_sync(~0u, q, m);
  }
  __syncthreads();  // the last call's readers are done
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = make_float2(p, q);
  __syncthreads();
  float2 s = part[0];
#pragma unroll
  for (int w = 1; w < kNormThreads / 32; ++w) {
    s.x += part[w].x;
    s.y += part[w].y;
  }
  return s;
}

template <typename Act, int NI>
__device__ __forceinline__ void row_load(const Tok& t, int64_t at, int D, float* v) {
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int d = i * kNormThreads + threadIdx.x;
    v[i] = d < D ? Num<Act>::to_f(static_cast<const Act*>(t.p)[at + d]) : 0.0f;
  }
}

template <typename Act, int NI>
__device__ __forceinline__ void row_store(const Tok& t, int64_t at, int D, const float* v) {
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int d = i * kNormThreads + threadIdx.x;
    if (d < D) static_cast<Act*>(t.p)[at + d] = Num<Act>::from_f(v[i]);
  }
}

__device__ __forceinline__ int64_t row_offset(const Tok& t, int b, int l, int h) {
  return b * t.sb + l * t.sl + h * t.sh;
}

// x <- n, returns 1 / sqrt(variance + eps).
template <int NI>
__device__ __forceinline__ float normalise(const NormArgs& a, float* x) {
  if (a.center) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i) s += x[i];
    const float m = cta_sum(s, 0.0f).x * a.inv_d;
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (i * kNormThreads + (int)threadIdx.x < a.D) x[i] -= m;
  }
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < NI; ++i) s = fmaf(x[i], x[i], s);
  const float rstd = 1.0f / sqrtf(cta_sum(s, 0.0f).x * a.inv_d + a.eps);
#pragma unroll
  for (int i = 0; i < NI; ++i) x[i] *= rstd;
  return rstd;
}

template <typename Act, int NI>
__global__ void __launch_bounds__(kNormThreads) norm_kernel(NormArgs a) {
  const int64_t rows = (int64_t)a.B * a.L * a.H;
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const int h = (int)(r % a.H), l = (int)(r / a.H % a.L), b = (int)(r / a.H / a.L);
    if (l >= seq_len(a.lens, b, a.L)) continue;
    float x[NI], z[NI];
    row_load<Act, NI>(a.x, row_offset(a.x, b, l, h), a.D, x);
    if (a.z.p) row_load<Act, NI>(a.z, row_offset(a.z, b, l, h), a.D, z);
    normalise<NI>(a, x);
    const int base = a.per_channel ? h * a.D : 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int d = i * kNormThreads + threadIdx.x;
      if (d >= a.D) continue;
      float u = x[i] * a.w[base + d];
      if (a.bias) u += a.bias[base + d];
      x[i] = a.z.p ? u * act_slope(a.activation, z[i]).x : act_slope(a.activation, u).x;
    }
    row_store<Act, NI>(a.y, row_offset(a.y, b, l, h), a.D, x);
  }
}

// CTA = (part, head): it walks every parts-th token of its head and leaves its sums of du n and
// du in partials[part][head][2][D].
template <typename Act, int NI>
__global__ void __launch_bounds__(kNormThreads) norm_backward_kernel(NormArgs a, int parts) {
  const int h = blockIdx.x % a.H, part = blockIdx.x / a.H;
  const int base = a.per_channel ? h * a.D : 0;
  float w[NI], bias[NI], sw[NI], sb[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int d = i * kNormThreads + threadIdx.x;
    w[i] = d < a.D ? a.w[base + d] : 0.0f;
    bias[i] = a.bias && d < a.D ? a.bias[base + d] : 0.0f;
    sw[i] = sb[i] = 0.0f;
  }
  for (int64_t t = part; t < (int64_t)a.B * a.L; t += parts) {
    const int b = (int)(t / a.L), l = (int)(t % a.L);
    if (l >= seq_len(a.lens, b, a.L)) continue;
    float x[NI], z[NI], dy[NI];
    row_load<Act, NI>(a.x, row_offset(a.x, b, l, h), a.D, x);
    row_load<Act, NI>(a.grad_y, row_offset(a.grad_y, b, l, h), a.D, dy);
    if (a.z.p) row_load<Act, NI>(a.z, row_offset(a.z, b, l, h), a.D, z);
    const float rstd = normalise<NI>(a, x);
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const float u = fmaf(x[i], w[i], bias[i]);
      const float2 f = act_slope(a.activation, a.z.p ? z[i] : u);
      const float du = dy[i] * (a.z.p ? f.x : f.y);
      z[i] = dy[i] * u * f.y;  // grad_z
      sw[i] = fmaf(du, x[i], sw[i]);
      sb[i] += du;
      dy[i] = du * w[i];  // dn
      s1 += dy[i];
      s2 = fmaf(dy[i], x[i], s2);
    }
    const float2 s = cta_sum(s1, s2);
    const float m1 = a.center ? s.x * a.inv_d : 0.0f, m2 = s.y * a.inv_d;
#pragma unroll
    for (int i = 0; i < NI; ++i) dy[i] = (dy[i] - m1 - x[i] * m2) * rstd;
    row_store<Act, NI>(a.grad_x, row_offset(a.grad_x, b, l, h), a.D, dy);
    if (a.z.p) row_store<Act, NI>(a.grad_z, row_offset(a.grad_z, b, l, h), a.D, z);
  }
  float* p = a.partials + (int64_t)blockIdx.x * 2 * a.D;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int d = i * kNormThreads + threadIdx.x;
    if (d < a.D) {
      p[d] = sw[i];
      p[a.D + d] = sb[i];
    }
  }
}

// grad_w and grad_bias from partials[parts][H][2][D]: 32 channels per CTA, the partial sums
// shared out over its 8 warps and added in the same order every time.
__global__ void __launch_bounds__(256) norm_reduce_kernel(NormArgs a, int parts);

}  // namespace gdnq
