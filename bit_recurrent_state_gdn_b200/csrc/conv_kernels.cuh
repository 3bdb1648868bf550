// Causal depthwise convolution over K tokens, with SiLU, and its gradients
// (include/gdnq_layer.h).
//
// A thread holds V neighbouring channels and walks a run of tokens, the last K inputs (and,
// backward, the last K gradients dp of the sums p) in registers, so that every array is read and
// written once but for the K - 1 tokens before (backward, also behind) a run. Backward p is formed
// again from x, and input s = t - K + 1 has all its gradient, sum_j w_j dp_{t-j}, when token t is
// done; a run forms the dp of the K - 1 tokens behind it too, without adding them to grad_w.
//
// Bound by HBM, and by latency at the two CTAs per SM that the windows' registers leave: rows come
// K at a time through a ring in shared memory, in slots of the thread's own (no barrier in the
// loop). bf16, K = 4, of 6452 GB/s: forward 8 x 4096 channels x 4096 tokens 97 us, 5.5 TB/s;
// backward 4 sequences 89 us, 4.5 TB/s; one token of 1024 sequences 16 us, 4.1 TB/s.
#pragma once

#include <type_traits>

#include "layer_util.cuh"

namespace gdnq {

constexpr int kConvThreads = 256;

// How a launch is shared out: runs per sequence, tokens of a run; backward also the CTAs that
// take the same channels.
struct ConvSplit {
  int runs, run_tokens, columns, parts;
};

// V elements at p as pairs (V even), or one and a zero.
template <typename Act, int V>
struct Vec {
  static constexpr int P = (V + 1) / 2;
  static __device__ __forceinline__ void get(const void* p, F2* f) {
    if constexpr (V == 1) {
      f[0] = f2(Num<Act>::to_f(*static_cast<const Act*>(p)), 0.0f);
    } else if constexpr (sizeof(Act) == 4 && V == 4) {
      const float4 t = *static_cast<const float4*>(p);
      f[0] = f2(t.x, t.y);
      f[1] = f2(t.z, t.w);
    } else if constexpr (sizeof(Act) == 4) {
      const float2 t = *static_cast<const float2*>(p);
      f[0] = f2(t.x, t.y);
    } else {
      uint32_t t[V / 2];
      if constexpr (V == 8) *reinterpret_cast<uint4*>(t) = *static_cast<const uint4*>(p);
      if constexpr (V == 4) *reinterpret_cast<uint2*>(t) = *static_cast<const uint2*>(p);
      if constexpr (V == 2) t[0] = *static_cast<const uint32_t*>(p);
#pragma unroll
      for (int i = 0; i < P; ++i) f[i] = f2(bf16_lo(t[i]), bf16_hi(t[i]));
    }
  }
  static __device__ __forceinline__ void put(void* p, const F2* f) {
    float lo, hi;
    if constexpr (V == 1) {
      f2_get(f[0], lo, hi);
      *static_cast<Act*>(p) = Num<Act>::from_f(lo);
    } else if constexpr (sizeof(Act) == 4 && V == 4) {
      float4 t;
      f2_get(f[0], t.x, t.y);
      f2_get(f[1], t.z, t.w);
      *static_cast<float4*>(p) = t;
    } else if constexpr (sizeof(Act) == 4) {
      float2 t;
      f2_get(f[0], t.x, t.y);
      *static_cast<float2*>(p) = t;
    } else {
      uint32_t t[V / 2];
#pragma unroll
      for (int i = 0; i < P; ++i) {
        f2_get(f[i], lo, hi);
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        t[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
      if constexpr (V == 8) *static_cast<uint4*>(p) = *reinterpret_cast<uint4*>(t);
      if constexpr (V == 4) *static_cast<uint2*>(p) = *reinterpret_cast<uint2*>(t);
      if constexpr (V == 2) *static_cast<uint32_t*>(p) = t[0];
    }
  }
};

// Rows of N arrays, K at a time from token t on; rows at or behind `end` read as zero.
//
// RowsInShared: V elements are 8 or 16 aligned bytes, S - 1 blocks ahead.
template <typename Act, int V_, int K, int N, int S>
struct RowsInShared {
  static constexpr int V = V_, kPiece = V * (int)sizeof(Act), kSlot = kConvThreads * kPiece;
  static constexpr int kBytes = S * N * K * kSlot;
  const Act* p[N];
  int64_t sl[N];
  uint32_t ring;
  const uint8_t* now;
  int t, end, fill, read;
  __device__ __forceinline__ RowsInShared(uint8_t* shared)
      : ring(smem_u32(shared) + threadIdx.x * kPiece), now(shared + threadIdx.x * kPiece) {}
  __device__ __forceinline__ void start(const Act* const (&from)[N], const int64_t (&stride)[N],
                                        int first, int end_) {
#pragma unroll
    for (int n = 0; n < N; ++n) p[n] = from[n], sl[n] = stride[n];
    t = first;
    end = end_;
    fill = 0;
    read = 0;
#pragma unroll
    for (int i = 0; i < S - 1; ++i) fetch();
  }
  __device__ __forceinline__ void fetch() {
    const uint32_t to = ring + (uint32_t)(fill * N * K * kSlot);
    const bool whole = t + K <= end;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const Act* row = p[n] + t * sl[n];
      if (whole) {
#pragma unroll
        for (int j = 0; j < K; ++j, row += sl[n])
          async_piece<kPiece>(to + (uint32_t)((n * K + j) * kSlot), row);
      } else {
#pragma unroll
        for (int j = 0; j < K; ++j, row += sl[n])
          async_piece<kPiece>(to + (uint32_t)((n * K + j) * kSlot), t + j < end ? row : p[n], t + j < end);
      }
    }
    asm volatile("cp.async.commit_group;\n" ::: "memory");
    t += K;
    fill = fill + 1 == S ? 0 : fill + 1;
  }
  // the next block is there
  __device__ __forceinline__ void take() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(S - 2) : "memory");
  }
  __device__ __forceinline__ void get(int n, int j, F2* f) const {
    Vec<Act, V>::get(now + (read * N * K + n * K + j) * kSlot, f);
  }
  // the block has been read
  __device__ __forceinline__ void done() {
    read = read + 1 == S ? 0 : read + 1;
    fetch();
  }
  __device__ __forceinline__ void finish() { asm volatile("cp.async.wait_all;\n" ::: "memory"); }
};

// RowsInRegisters: single elements at any alignment, one block ahead.
template <typename Act, int K, int N>
struct RowsInRegisters {
  static constexpr int V = 1, kBytes = 0;
  const Act* p[N];
  int64_t sl[N];
  int t, end;
  Act next[N][K], now[N][K];
  __device__ __forceinline__ RowsInRegisters(uint8_t*) {}
  __device__ __forceinline__ void start(const Act* const (&from)[N], const int64_t (&stride)[N],
                                        int first, int end_) {
#pragma unroll
    for (int n = 0; n < N; ++n) p[n] = from[n], sl[n] = stride[n];
    t = first;
    end = end_;
    fetch();
  }
  __device__ __forceinline__ void fetch() {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int j = 0; j < K; ++j)
        next[n][j] = t + j < end ? p[n][(t + j) * sl[n]] : Num<Act>::from_f(0.0f);
    t += K;
  }
  __device__ __forceinline__ void take() {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int j = 0; j < K; ++j) now[n][j] = next[n][j];
    fetch();
  }
  __device__ __forceinline__ void get(int n, int j, F2* f) const {
    f[0] = f2(Num<Act>::to_f(now[n][j]), 0.0f);
  }
  __device__ __forceinline__ void done() {}
  __device__ __forceinline__ void finish() {}
};

// Input of token t < 0 of channels c ..: what the state holds.
template <typename Act, int V, int K>
__device__ __forceinline__ void state_get(const void* state, const ConvArgs& a, int b, int c, int t, F2* f) {
  if (state == nullptr) {
#pragma unroll
    for (int i = 0; i < Vec<Act, V>::P; ++i) f[i] = f2_all(0.0f);
    return;
  }
  Vec<Act, V>::get(static_cast<const Act*>(state) + ((int64_t)b * (K - 1) + t + K - 1) * a.C + c, f);
}

template <typename Act, int V, int K>
__device__ __forceinline__ void state_put(void* state, const ConvArgs& a, int b, int c, int t, const F2* f) {
  Vec<Act, V>::put(static_cast<Act*>(state) + ((int64_t)b * (K - 1) + t + K - 1) * a.C + c, f);
}

// w[c + v][j] as pairs over v: V K floats in a row.
template <int V, int K>
__device__ __forceinline__ void taps(const ConvArgs& a, int c, F2 (&w)[K][(V + 1) / 2],
                                     F2 (&bias)[(V + 1) / 2]) {
  float flat[V * K + K] = {};
  const float* p = a.w + (int64_t)c * K;
  if (V % 4 == 0 && reinterpret_cast<uintptr_t>(a.w) % 16 == 0) {
#pragma unroll
    for (int i = 0; i < V * K / 4; ++i) {
      const float4 t = reinterpret_cast<const float4*>(p)[i];
      flat[4 * i] = t.x, flat[4 * i + 1] = t.y, flat[4 * i + 2] = t.z, flat[4 * i + 3] = t.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V * K; ++i) flat[i] = p[i];
  }
#pragma unroll
  for (int i = 0; i < (V + 1) / 2; ++i) {
#pragma unroll
    for (int j = 0; j < K; ++j) w[j][i] = f2(flat[2 * i * K + j], flat[(2 * i + 1) * K + j]);
    bias[i] = f2_all(0.0f);
    if (a.bias) bias[i] = f2(a.bias[c + 2 * i], V > 1 ? a.bias[c + 2 * i + (V > 1)] : 0.0f);
  }
}

template <typename Act, int K, bool SILU, class Rows, int MINB>
__global__ void __launch_bounds__(kConvThreads, MINB) conv_kernel(ConvArgs a, ConvSplit split) {
  constexpr int V = Rows::V, P = Vec<Act, V>::P;
  extern __shared__ __align__(128) uint8_t rings[];
  // a thread keeps its channels, whose taps it reads once, and takes every split.parts-th run
  const int64_t i = (int64_t)blockIdx.x * kConvThreads + threadIdx.x;
  if (i >= (int64_t)split.parts * split.columns) return;
  const int c = (int)(i % split.columns) * V, hd = c / a.D, d = c % a.D;
  F2 w[K][P], bias[P];
  taps<V, K>(a, c, w, bias);
  Rows rows(rings);
  for (int64_t r = i / split.columns; r < (int64_t)a.B * split.runs; r += split.parts) {
    const int b = (int)(r / split.runs), t0 = (int)(r % split.runs) * split.run_tokens;
    const int len = seq_len(a.lens, b, a.L), t1 = min(t0 + split.run_tokens, len);
    if (t0 > 0 && t0 >= len) continue;
    const Act* x = static_cast<const Act*>(a.x.p) + channel_offset(a.x, b, hd, d);
    Act* y = static_cast<Act*>(a.y.p) + channel_offset(a.y, b, hd, d) + t0 * a.y.sl;
    const Act* const from[1] = {x};
    const int64_t stride[1] = {a.x.sl};
    if (t0 < t1) rows.start(from, stride, t0, t1);
    F2 win[K][P];  // win[i]: the input of the last token t with (t - t0) % K == i
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      const int t = t0 - (K - 1) + j;
      if (t >= 0)
        Vec<Act, V>::get(x + t * a.x.sl, win[j + 1]);
      else
        state_get<Act, V, K>(a.state_in, a, b, c, t, win[j + 1]);
    }
    // What the sequence leaves. In one run of K - 1 tokens or more the window has it in the end.
    // Else the run that begins the sequence hands it on: it alone reads state_in, which state_out
    // may be.
    const bool from_window = split.runs == 1 && len >= K - 1;
    if (a.state_out && t0 == 0 && !from_window) {
      F2 keep[K - 1][P];
#pragma unroll
      for (int j = 0; j < K - 1; ++j) {
        const int t = len - (K - 1) + j;
        if (t >= 0)
          Vec<Act, V>::get(x + t * a.x.sl, keep[j]);
        else
          state_get<Act, V, K>(a.state_in, a, b, c, t, keep[j]);
      }
#pragma unroll
      for (int j = 0; j < K - 1; ++j) state_put<Act, V, K>(a.state_out, a, b, c, j - (K - 1), keep[j]);
    }
    // a block of K tokens; inside the run its stores need no conditions, which keeps the K tokens
    // in one stretch of code
    auto block = [&](int t, auto inside) {
#pragma unroll
      for (int u = 0; u < K; ++u) {
        rows.get(0, u, win[u]);
        F2 out[P];
#pragma unroll
        for (int e = 0; e < P; ++e) {
          F2 p = bias[e];
#pragma unroll
          for (int j = 0; j < K; ++j) p = f2_fma(w[j][e], win[(u + 1 + j) % K][e], p);
          F2 slope;
          act_pair<SILU ? GDN_ACT_SILU : GDN_ACT_NONE, false>(p, out[e], slope);
        }
        if (decltype(inside)::value || t + u < t1) {
          Vec<Act, V>::put(y, out);
          y += a.y.sl;
          if (!decltype(inside)::value && a.state_out && from_window && t + u >= len - (K - 1))
            state_put<Act, V, K>(a.state_out, a, b, c, t + u - len, win[u]);
        }
      }
    };
    for (int t = t0; t < t1; t += K) {
      rows.take();
      if (t + 2 * K <= t1)
        block(t, std::true_type());
      else
        block(t, std::false_type());
      rows.done();
    }
    rows.finish();
  }
}

// One token: the inputs that the state holds and x, U sequences at a time so that their loads are
// under way together; as they lie in memory until they are used, which also hands them on exactly.
template <typename Act, int K, bool SILU, int V, int U, int MINB>
__global__ void __launch_bounds__(kConvThreads, MINB) conv_step_kernel(ConvArgs a, ConvSplit split) {
  constexpr int P = Vec<Act, V>::P;
  struct alignas(V * sizeof(Act)) Raw {
    Act e[V];
  };
  const int64_t i = (int64_t)blockIdx.x * kConvThreads + threadIdx.x;
  if (i >= (int64_t)split.parts * split.columns) return;
  const int c = (int)(i % split.columns) * V, hd = c / a.D, d = c % a.D;
  F2 w[K][P], bias[P];
  taps<V, K>(a, c, w, bias);
  for (int64_t first = i / split.columns; first < a.B; first += (int64_t)split.parts * U) {
    Raw in[U][K];
    bool there[U], token[U];
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int64_t b = first + (int64_t)q * split.parts;
      there[q] = b < a.B;
      token[q] = there[q] && (a.lens == nullptr || a.lens[b] > 0);
#pragma unroll
      for (int j = 0; j < K; ++j) in[q][j] = Raw{};
      if (there[q] && a.state_in) {
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
          in[q][j] = *reinterpret_cast<const Raw*>(static_cast<const Act*>(a.state_in) +
                                                   (b * (K - 1) + j) * a.C + c);
      }
      if (token[q])
        in[q][K - 1] = *reinterpret_cast<const Raw*>(static_cast<const Act*>(a.x.p) +
                                                     channel_offset(a.x, (int)b, hd, d));
    }
#pragma unroll
    for (int q = 0; q < U; ++q) {
      if (!there[q]) continue;
      const int64_t b = first + (int64_t)q * split.parts;
      Act* out_state = static_cast<Act*>(a.state_out) + b * (K - 1) * a.C + c;
      if (token[q]) {
        if (a.state_out) {
#pragma unroll
          for (int j = 0; j < K - 1; ++j) *reinterpret_cast<Raw*>(out_state + (int64_t)j * a.C) = in[q][j + 1];
        }
        F2 p[P];
#pragma unroll
        for (int e = 0; e < P; ++e) p[e] = bias[e];
#pragma unroll
        for (int j = 0; j < K; ++j) {
          F2 v[P];
          Vec<Act, V>::get(&in[q][j], v);
#pragma unroll
          for (int e = 0; e < P; ++e) p[e] = f2_fma(w[j][e], v[e], p[e]);
        }
#pragma unroll
        for (int e = 0; e < P; ++e) {
          F2 slope, v = p[e];
          act_pair<SILU ? GDN_ACT_SILU : GDN_ACT_NONE, false>(v, p[e], slope);
        }
        Vec<Act, V>::put(static_cast<Act*>(a.y.p) + channel_offset(a.y, (int)b, hd, d), p);
      } else if (a.state_out) {
#pragma unroll
        for (int j = 0; j < K - 1; ++j) *reinterpret_cast<Raw*>(out_state + (int64_t)j * a.C) = in[q][j];
      }
    }
  }
}

// CTA = TX columns x TY runs at a time; its sums of dp x and dp go to partials[part][K + 1][C].
template <typename Act, int K, bool SILU, class Rows, int TX, int MINB>
__global__ void __launch_bounds__(kConvThreads, MINB) conv_backward_kernel(ConvArgs a, ConvSplit split) {
  constexpr int V = Rows::V, P = Vec<Act, V>::P, TY = kConvThreads / TX;
  extern __shared__ __align__(128) uint8_t rings[];
  let_next_launch();
  const int tx = threadIdx.x % TX, ty = threadIdx.x / TX;
  const int slabs = (split.columns + TX - 1) / TX;
  const int slab = (int)(blockIdx.x % (unsigned)slabs), part = (int)(blockIdx.x / (unsigned)slabs);
  const int column = slab * TX + tx, c = column * V;
  F2 w[K][P], bias[P], dw[K][P], db[P];
#pragma unroll
  for (int e = 0; e < P; ++e) {
    db[e] = f2_all(0.0f);
#pragma unroll
    for (int j = 0; j < K; ++j) dw[j][e] = f2_all(0.0f);
  }
  Rows rows(rings);
  if (column < split.columns) {
    const int hd = c / a.D, d = c % a.D;
    taps<V, K>(a, c, w, bias);
    // a CTA's runs lie far apart: in a padded batch every CTA has its share of the runs behind the
    // sequences' ends (4 sequences, 88 % of the tokens: 92 us with neighbouring runs)
    for (int64_t r = (int64_t)ty * split.parts + part; r < (int64_t)a.B * split.runs;
         r += (int64_t)split.parts * TY) {
      const int b = (int)(r / split.runs), t0 = (int)(r % split.runs) * split.run_tokens;
      const int len = seq_len(a.lens, b, a.L), t1 = min(t0 + split.run_tokens, len);
      if (t0 > 0 && t0 >= len) continue;
      const Act* x = static_cast<const Act*>(a.x.p) + channel_offset(a.x, b, hd, d);
      const Act* gy = static_cast<const Act*>(a.grad_y.p) + channel_offset(a.grad_y, b, hd, d);
      Act* gx = static_cast<Act*>(a.grad_x.p) + channel_offset(a.grad_x, b, hd, d) +
                (t0 - (K - 1)) * a.grad_x.sl;  // input s = t - K + 1, from t = t0 on
      const Act* const from[2] = {x, gy};
      const int64_t stride[2] = {a.x.sl, a.grad_y.sl};
      rows.start(from, stride, t0, min(t1 + K - 1, len));
      F2 win[K][P], dp[K][P];  // of the last token t with (t - t0) % K == i
#pragma unroll
      for (int j = 0; j < K - 1; ++j) {
        const int t = t0 - (K - 1) + j;
        if (t >= 0)
          Vec<Act, V>::get(x + t * a.x.sl, win[j + 1]);
        else
          state_get<Act, V, K>(a.state_in, a, b, c, t, win[j + 1]);
#pragma unroll
        for (int e = 0; e < P; ++e) dp[j + 1][e] = f2_all(0.0f);
      }
      // a block of K tokens; inside the run its stores need no conditions, which keeps the K
      // tokens in one stretch of code (8 heads of 128 x 16384 tokens: 112 us without this)
      auto block = [&](int t, auto inside) {
        constexpr bool kInside = decltype(inside)::value;
#pragma unroll
        for (int u = 0; u < K; ++u) {
          F2 dy[P], g[P];
          rows.get(0, u, win[u]);
          rows.get(1, u, dy);
#pragma unroll
          for (int e = 0; e < P; ++e) {
            F2 p = bias[e];
#pragma unroll
            for (int j = 0; j < K; ++j) p = f2_fma(w[j][e], win[(u + 1 + j) % K][e], p);
            F2 v, slope;
            act_pair<SILU ? GDN_ACT_SILU : GDN_ACT_NONE, true>(p, v, slope);
            dp[u][e] = f2_mul(dy[e], slope);
            // token t + u - j has dp[(u - j) mod K]
            g[e] = f2_mul(w[0][e], dp[u][e]);
#pragma unroll
            for (int j = 1; j < K; ++j) g[e] = f2_fma(w[j][e], dp[(u + K - j) % K][e], g[e]);
          }
          if (kInside || t + u < t1) {  // dp behind the run is another run's, or none's
#pragma unroll
            for (int e = 0; e < P; ++e) {
              db[e] = f2_add(db[e], dp[u][e]);
#pragma unroll
              for (int j = 0; j < K; ++j) dw[j][e] = f2_fma(dp[u][e], win[(u + 1 + j) % K][e], dw[j][e]);
            }
          }
          if constexpr (kInside) {
            Vec<Act, V>::put(gx, g);
          } else {
            const int s = t + u - (K - 1), behind = t + u - len;
            if (t + u < t1 + K - 1 && (s >= t0 || t0 == 0)) {
              if (behind >= 0 && a.grad_state_out) {
                F2 more[P];
                state_get<Act, V, K>(a.grad_state_out, a, b, c, behind - (K - 1), more);
#pragma unroll
                for (int e = 0; e < P; ++e) g[e] = f2_add(g[e], more[e]);
              }
              if (s >= 0)
                Vec<Act, V>::put(gx, g);
              else if (a.grad_state_in)
                state_put<Act, V, K>(a.grad_state_in, a, b, c, s, g);
            }
          }
          gx += a.grad_x.sl;
        }
      };
      for (int t = t0; t < t1 + K - 1; t += K) {
        rows.take();
        if (t > t0 && t + K <= t1)
          block(t, std::true_type());
        else
          block(t, std::false_type());
        rows.done();
      }
      rows.finish();
    }
  }
  // the CTA's sums over its runs, in order
  __syncthreads();
  float* sums = reinterpret_cast<float*>(rings);  // [TY][K + 1][TX V]
  constexpr int kWide = TX * V;
#pragma unroll
  for (int j = 0; j <= K; ++j) {
#pragma unroll
    for (int e = 0; e < P; ++e) {
      float lo, hi;
      f2_get(j < K ? dw[j < K ? j : 0][e] : db[e], lo, hi);
      float* at = sums + (ty * (K + 1) + j) * kWide + tx * V + 2 * e;
      at[0] = lo;
      if constexpr (V > 1) at[1] = hi;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < (K + 1) * kWide; i += kConvThreads) {
    const int64_t channel = (int64_t)slab * kWide + i % kWide;
    if (channel >= a.C) continue;
    float s = 0.0f;
    for (int q = 0; q < TY; ++q) s += sums[q * (K + 1) * kWide + i];
    a.partials[((int64_t)part * (K + 1) + i / kWide) * a.C + channel] = s;
  }
}

template <int K, int TX, class Rows>
constexpr int conv_backward_shared() {
  constexpr int sums = kConvThreads * (K + 1) * Rows::V * 4;
  return Rows::kBytes > sums ? Rows::kBytes : sums;
}

}  // namespace gdnq
