// Group norm over each head's channels with an activation or a gate, and its gradients
// (include/gdnq_layer.h).
//
// Mathematics. A row is one head of one token. Its D channels are read once into registers; the
// mean and the mean square of what is left of it are two sums over the row's lanes, in that order,
// so that no difference of large squares is taken. Backward the row is normed again from x (cheaper
// than reading kept statistics would be to write) and the two row sums of dn and dn n follow.
//
// Split. LANES lanes of a warp hold a row, a CTA holds 256 / LANES rows at a time: HB neighbouring
// heads (a power of two) of TB tokens. A lane keeps its head, so that the weights stay in registers
// and the sums for their gradients do too, and walks tokens; these sums are joined over the CTA
// in shared memory, written as partial sums, and added by a second kernel in a fixed order.
//
// Bound by HBM, and close to it by instructions: rows come through a ring in shared memory, S rows
// ahead, each lane copying the pieces that it will read (no barrier in the loop). bf16, rows of 128
// with a gate, of 6452 GB/s: forward 8 x 32 x 4096 tokens 136 us, 5.9 TB/s (24 instructions per
// element); backward 4 x 32 x 4096 119 us, 5.6 TB/s (38); in long runs over changing inputs, which the
// power limit slows down, the forward pass takes 148 us.
#pragma once

#include <type_traits>

#include "layer_util.cuh"

namespace gdnq {

constexpr int kNormThreads = 256;

// How rows are shared out over a launch; made by norm_plan.
struct NormSplit {
  int hb_log, heads_of_blocks, parts;  // blocks of HB heads; CTAs per block of heads
};

// act(u) and act'(u).
__device__ __forceinline__ float2 act_slope(int activation, float u) {
  if (activation == GDN_ACT_NONE) return make_float2(u, 1.0f);
  const float q = sigmoidf(u);
  if (activation == GDN_ACT_SIGMOID) return make_float2(q, q * (1.0f - q));
  return make_float2(u * q, q * fmaf(u, 1.0f - q, 1.0f));
}

// V elements of Act at p, as floats.
template <typename Act, int V>
__device__ __forceinline__ void piece_get(const void* p, float* f) {
  if constexpr (V == 1) {
    f[0] = Num<Act>::to_f(*static_cast<const Act*>(p));
  } else if constexpr (sizeof(Act) == 4) {
    if constexpr (V == 4) {
      const float4 t = *static_cast<const float4*>(p);
      f[0] = t.x, f[1] = t.y, f[2] = t.z, f[3] = t.w;
    } else {
      const float2 t = *static_cast<const float2*>(p);
      f[0] = t.x, f[1] = t.y;
    }
  } else {
    uint32_t t[V / 2];
    if constexpr (V == 8) *reinterpret_cast<uint4*>(t) = *static_cast<const uint4*>(p);
    if constexpr (V == 4) *reinterpret_cast<uint2*>(t) = *static_cast<const uint2*>(p);
    if constexpr (V == 2) t[0] = *static_cast<const uint32_t*>(p);
#pragma unroll
    for (int e = 0; e < V / 2; ++e) f[2 * e] = bf16_lo(t[e]), f[2 * e + 1] = bf16_hi(t[e]);
  }
}

template <typename Act, int V>
__device__ __forceinline__ void piece_put(void* p, const float* f) {
  if constexpr (V == 1) {
    *static_cast<Act*>(p) = Num<Act>::from_f(f[0]);
  } else if constexpr (sizeof(Act) == 4) {
    if constexpr (V == 4)
      *static_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    else
      *static_cast<float2*>(p) = make_float2(f[0], f[1]);
  } else {
    uint32_t t[V / 2];
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
      t[e] = *reinterpret_cast<const uint32_t*>(&h);
    }
    if constexpr (V == 8) *static_cast<uint4*>(p) = *reinterpret_cast<uint4*>(t);
    if constexpr (V == 4) *static_cast<uint2*>(p) = *reinterpret_cast<uint2*>(t);
    if constexpr (V == 2) *static_cast<uint32_t*>(p) = t[0];
  }
}

// A lane's walk over the tokens of its head, every step-th one; an Offset follows it through one
// array without multiplications.
struct Walk {
  int b, l, step_b, step_l;
  int64_t left, step;  // tokens from here to the end, this one included; <= 0 behind it
  bool wrapped;        // by the last next()
  __device__ __forceinline__ Walk(int64_t first, int64_t step_, int64_t tokens, int L)
      : b((int)(first / L)), l((int)(first % L)), step_b((int)(step_ / L)), step_l((int)(step_ % L)),
        left(tokens - first), step(step_), wrapped(false) {}
  __device__ __forceinline__ void next(int L) {
    b += step_b;
    l += step_l;
    wrapped = l >= L;
    if (wrapped) {
      l -= L;
      ++b;
    }
    left -= step;
  }
  __device__ __forceinline__ bool live(const int32_t* lens, int L) const {
    return left > 0 && (lens == nullptr || l < seq_len(lens, b, L));
  }
};

template <typename Act>
struct Offset {
  Act* p;
  int64_t step, wrap;
  __device__ __forceinline__ Offset(const Tok& t, const Walk& w, int h, int d, int L)
      : p(static_cast<Act*>(t.p) + (w.b * t.sb + w.l * t.sl + h * t.sh + d)),
        step(w.step_b * t.sb + w.step_l * t.sl), wrap(t.sb - L * t.sl) {}
  __device__ __forceinline__ void next(const Walk& w) {
    p += step;
    if (w.wrapped) p += wrap;
  }
};

// The pieces of NI x LANES x V channels that one lane reads of each array of a row, N arrays.
//
// PiecesInShared: pieces of 4, 8 or 16 aligned bytes, S - 1 rows ahead, in slots of the lane's own.
// WHOLE: warps whose pieces are all there copy them without conditions. Forward that takes 8 x 32 x
// 4096 gated rows of 128 from 5668 to 5875 GB/s (a padded batch from 5260 to 5076); backward, where
// the second path costs registers, from 5630 to 5429, so it is without.
template <typename Act, int V_, int LANES_, int NI_, int N, int S, bool WHOLE>
struct PiecesInShared {
  static constexpr int LANES = LANES_, NI = NI_, V = V_, kPiece = V * (int)sizeof(Act);
  static constexpr int kSlot = kNormThreads * kPiece;
  static constexpr int kBytes = S * N * NI * kSlot;
  uint32_t ring;
  const uint8_t* now;
  int fill = 0, read = 0;
  __device__ __forceinline__ PiecesInShared(uint8_t* shared)
      : ring(smem_u32(shared) + threadIdx.x * kPiece), now(shared + threadIdx.x * kPiece) {}
  // from[n] points at the lane's first piece of array n, ok[i] says whether piece i is there: a
  // copy of no bytes fills its slot with zeros, so that the row is read without conditions
  __device__ __forceinline__ void fetch(const Act* const (&from)[N], const Act* const (&base)[N],
                                        const bool (&ok)[NI]) {
    const uint32_t to = ring + (uint32_t)(fill * N * NI * kSlot);
    bool all = WHOLE;
#pragma unroll
    for (int i = 0; i < NI; ++i) all = all && ok[i];
    if (WHOLE && __all_sync(~0u, all)) {
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < NI; ++i)
          async_piece<kPiece>(to + (uint32_t)((n * NI + i) * kSlot), from[n] + i * LANES * V);
    } else {
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < NI; ++i)
          async_piece<kPiece>(to + (uint32_t)((n * NI + i) * kSlot),
                              ok[i] ? from[n] + i * LANES * V : base[n], ok[i]);
    }
    asm volatile("cp.async.commit_group;\n" ::: "memory");
    fill = fill + 1 == S ? 0 : fill + 1;
  }
  static constexpr int kAhead = S - 1;
  __device__ __forceinline__ void wait() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(S - 2) : "memory");
  }
  __device__ __forceinline__ void get(int n, int i, float* f) const {
    piece_get<Act, V>(now + (read * N * NI + n * NI + i) * kSlot, f);
  }
  __device__ __forceinline__ void done() { read = read + 1 == S ? 0 : read + 1; }
};

// PiecesInRegisters: single elements at any alignment, one row ahead.
template <typename Act, int LANES_, int NI_, int N>
struct PiecesInRegisters {
  static constexpr int LANES = LANES_, NI = NI_, V = 1, kBytes = 0, kAhead = 1;
  Act next[N][NI], now[N][NI];
  __device__ __forceinline__ PiecesInRegisters(uint8_t*) {}
  __device__ __forceinline__ void fetch(const Act* const (&from)[N], const Act* const (&)[N],
                                        const bool (&ok)[NI]) {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int i = 0; i < NI; ++i)
        next[n][i] = ok[i] ? from[n][i * LANES] : Num<Act>::from_f(0.0f);
  }
  __device__ __forceinline__ void wait() {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int i = 0; i < NI; ++i) now[n][i] = next[n][i];
  }
  __device__ __forceinline__ void get(int n, int i, float* f) const { f[0] = Num<Act>::to_f(now[n][i]); }
  __device__ __forceinline__ void done() {}
};

template <int LANES>
__device__ __forceinline__ float lanes_sum(float s) {
#pragma unroll
  for (int m = LANES / 2; m; m >>= 1) s += __shfl_xor_sync(~0u, s, m);
  return s;
}

__device__ __forceinline__ int64_t row_offset(const Tok& t, int b, int l, int h) {
  return b * t.sb + l * t.sl + h * t.sh;
}

__device__ __forceinline__ float f2_sum(F2 a) {
  float lo, hi;
  f2_get(a, lo, hi);
  return lo + hi;
}

// What the kernels share: the lane's place, and the norm of a row.
template <class P>
struct NormLane {
  // a lane's channels two by two (the second of an only one is 0): channel c = i V + v is half
  // c % 2 of pair c / 2
  static constexpr int LANES = P::LANES, NI = P::NI, V = P::V, E = (NI * V + 1) / 2;
  int sub, h, hb, tb, part, first_head;
  bool ok[NI];  // the lane's head exists and its pieces lie within D
  __device__ __forceinline__ NormLane(const NormArgs& a, const NormSplit& s) {
    const int group = threadIdx.x / LANES;
    sub = threadIdx.x % LANES;
    hb = 1 << s.hb_log;
    tb = kNormThreads / LANES >> s.hb_log;
    first_head = (int)(blockIdx.x % (unsigned)s.heads_of_blocks) * hb;
    part = (int)(blockIdx.x / (unsigned)s.heads_of_blocks);
    h = first_head + group % hb;
#pragma unroll
    for (int i = 0; i < NI; ++i) ok[i] = h < a.H && (i * LANES + sub) * V < a.D;
  }
  __device__ __forceinline__ void weights(const NormArgs& a, const float* w, F2* f) const {
    const float* p = w + (a.per_channel ? (int64_t)h * a.D : 0);
    float flat[2 * E] = {};
#pragma unroll
    for (int i = 0; i < NI; ++i) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (w && ok[i]) flat[i * V + v] = p[(i * LANES + sub) * V + v];
    }
    pack(flat, f);
  }
  static __device__ __forceinline__ void pack(const float* flat, F2* f) {
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = f2(flat[2 * e], flat[2 * e + 1]);
  }
  static __device__ __forceinline__ void unpack(const F2* f, float* flat) {
#pragma unroll
    for (int e = 0; e < E; ++e) f2_get(f[e], flat[2 * e], flat[2 * e + 1]);
  }
  // array n of the row, 0 where there is none
  static __device__ __forceinline__ void get(const P& pieces, int n, F2* f) {
    float flat[2 * E] = {};
#pragma unroll
    for (int i = 0; i < NI; ++i)
      pieces.get(n, i, flat + i * V);
    pack(flat, f);
  }
  template <typename Act>
  __device__ __forceinline__ void put(Act* p, bool live, const F2* f) const {
    float flat[2 * E];
    unpack(f, flat);
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (live && ok[i]) piece_put<Act, V>(p + i * LANES * V, flat + i * V);
  }
  // x <- n (0 where there is no channel); returns 1 / sqrt(variance + eps)
  __device__ __forceinline__ float normalise(const NormArgs& a, F2* x) const {
    if (a.center) {
      F2 s = x[0];
#pragma unroll
      for (int e = 1; e < E; ++e) s = f2_add(s, x[e]);
      const float m = -lanes_sum<LANES>(f2_sum(s)) * a.inv_d;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        constexpr int last = NI * V - 1;
        x[e] = f2_add(x[e], f2(ok[2 * e / V] ? m : 0.0f,
                               2 * e < last && ok[(2 * e < last ? 2 * e + 1 : 0) / V] ? m : 0.0f));
      }
    }
    F2 s = f2_mul(x[0], x[0]);
#pragma unroll
    for (int e = 1; e < E; ++e) s = f2_fma(x[e], x[e], s);
    const float rstd = rsqrtf(fmaf(lanes_sum<LANES>(f2_sum(s)), a.inv_d, a.eps));
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = f2_mul(x[e], f2_all(rstd));
    return rstd;
  }
};

// Calls f with the activation as a constant: one uniform branch per row.
template <class F>
__device__ __forceinline__ void with_activation(int activation, F f) {
  if (activation == GDN_ACT_SILU)
    f(std::integral_constant<int, GDN_ACT_SILU>());
  else if (activation == GDN_ACT_SIGMOID)
    f(std::integral_constant<int, GDN_ACT_SIGMOID>());
  else
    f(std::integral_constant<int, GDN_ACT_NONE>());
}

template <typename Act, bool GATE, class P, int MINB>
__global__ void __launch_bounds__(kNormThreads, MINB) norm_kernel(NormArgs a, NormSplit split) {
  using Lane = NormLane<P>;
  constexpr int N = GATE ? 2 : 1, NI = P::NI, V = P::V, E = Lane::E;
  extern __shared__ __align__(128) uint8_t rings[];
  const Lane q(a, split);
  F2 w[E], bias[E];
  q.weights(a, a.w, w);
  q.weights(a, a.bias, bias);
  P pieces(rings);
  const int64_t tokens = (int64_t)a.B * a.L, step = (int64_t)split.parts * q.tb;
  const int64_t first = (int64_t)q.part * q.tb, mine = threadIdx.x / P::LANES >> split.hb_log;
  Walk ahead(first + mine, step, tokens, a.L), at = ahead;
  Offset<Act> x_at(a.x, ahead, q.h, q.sub * V, a.L), z_at(a.z, ahead, q.h, q.sub * V, a.L);
  Offset<Act> y_at(a.y, at, q.h, q.sub * V, a.L);
  auto fetch = [&]() {
    const bool live = ahead.live(a.lens, a.L);
    bool there[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) there[i] = live && q.ok[i];
    const Act *from[N], *base[N];
    from[0] = x_at.p, base[0] = static_cast<const Act*>(a.x.p);
    if constexpr (GATE) from[1] = z_at.p, base[1] = static_cast<const Act*>(a.z.p);
    pieces.fetch(from, base, there);
    ahead.next(a.L);
    x_at.next(ahead);
    if constexpr (GATE) z_at.next(ahead);
  };
#pragma unroll
  for (int i = 0; i < P::kAhead; ++i) fetch();
  for (int64_t t = first; t < tokens; t += step) {
    pieces.wait();
    const bool live = at.live(a.lens, a.L);
    F2 x[E], z[E];
    Lane::get(pieces, 0, x);
    if constexpr (GATE) Lane::get(pieces, 1, z);
    pieces.done();
    fetch();
    if (__any_sync(~0u, live)) {  // not behind the ends of all of the warp's sequences
      q.normalise(a, x);
      with_activation(a.activation, [&](auto act) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const F2 u = f2_fma(x[e], w[e], bias[e]);
          F2 v, slope;
          act_pair<decltype(act)::value, false>(GATE ? z[e] : u, v, slope);
          x[e] = GATE ? f2_mul(u, v) : v;
        }
      });
      q.put(y_at.p, live, x);
    }
    at.next(a.L);
    y_at.next(at);
  }
  asm volatile("cp.async.wait_all;\n" ::: "memory");  // copies behind the last row
}

// Shared memory: the ring, then (the loop done) two floats for every channel that a lane holds.
template <class P>
constexpr int norm_backward_shared() {
  constexpr int sums = kNormThreads * P::NI * P::V * 8;
  return P::kBytes > sums ? P::kBytes : sums;
}

// Leaves its sums of du n and du at partials[CTA][2][D] (weights shared by the heads) or
// partials[part][head][2][D].
template <typename Act, bool GATE, class P, int MINB>
__global__ void __launch_bounds__(kNormThreads, MINB) norm_backward_kernel(NormArgs a, NormSplit split) {
  using Lane = NormLane<P>;
  constexpr int N = GATE ? 3 : 2, NI = P::NI, V = P::V, E = Lane::E, LANES = P::LANES;
  extern __shared__ __align__(128) uint8_t rings[];
  let_next_launch();
  const Lane q(a, split);
  F2 w[E], bias[E], sw[E], sb[E];
  q.weights(a, a.w, w);
  q.weights(a, a.bias, bias);
#pragma unroll
  for (int e = 0; e < E; ++e) sw[e] = sb[e] = f2_all(0.0f);
  P pieces(rings);
  const int64_t tokens = (int64_t)a.B * a.L, step = (int64_t)split.parts * q.tb;
  const int64_t first = (int64_t)q.part * q.tb, mine = threadIdx.x / LANES >> split.hb_log;
  Walk ahead(first + mine, step, tokens, a.L), at = ahead;
  Offset<Act> x_at(a.x, ahead, q.h, q.sub * V, a.L), z_at(a.z, ahead, q.h, q.sub * V, a.L);
  Offset<Act> dy_at(a.grad_y, ahead, q.h, q.sub * V, a.L);
  Offset<Act> dx_at(a.grad_x, at, q.h, q.sub * V, a.L), dz_at(a.grad_z, at, q.h, q.sub * V, a.L);
  auto fetch = [&]() {
    const bool live = ahead.live(a.lens, a.L);
    bool there[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) there[i] = live && q.ok[i];
    const Act *from[N], *base[N];
    from[0] = x_at.p, base[0] = static_cast<const Act*>(a.x.p);
    from[1] = dy_at.p, base[1] = static_cast<const Act*>(a.grad_y.p);
    if constexpr (GATE) from[2] = z_at.p, base[2] = static_cast<const Act*>(a.z.p);
    pieces.fetch(from, base, there);
    ahead.next(a.L);
    x_at.next(ahead);
    dy_at.next(ahead);
    if constexpr (GATE) z_at.next(ahead);
  };
#pragma unroll
  for (int i = 0; i < P::kAhead; ++i) fetch();
  for (int64_t t = first; t < tokens; t += step) {
    pieces.wait();
    const bool live = at.live(a.lens, a.L);
    F2 x[E], dy[E], z[E];
    Lane::get(pieces, 0, x);
    Lane::get(pieces, 1, dy);
    if constexpr (GATE) Lane::get(pieces, 2, z);
    pieces.done();
    fetch();
    if (__any_sync(~0u, live)) {  // not behind the ends of all of the warp's sequences
      const float rstd = q.normalise(a, x);
      F2 s1 = f2_all(0.0f), s2 = s1;
      with_activation(a.activation, [&](auto act) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const F2 u = f2_fma(x[e], w[e], bias[e]);
          F2 v, slope;
          act_pair<decltype(act)::value, true>(GATE ? z[e] : u, v, slope);
          const F2 du = f2_mul(dy[e], GATE ? v : slope);
          if constexpr (GATE) z[e] = f2_mul(f2_mul(dy[e], u), slope);  // grad_z
          sw[e] = f2_fma(du, x[e], sw[e]);
          sb[e] = f2_add(sb[e], du);
          dy[e] = f2_mul(du, w[e]);  // dn
          s1 = f2_add(s1, dy[e]);
          s2 = f2_fma(dy[e], x[e], s2);
        }
      });
      const float m1 = a.center ? lanes_sum<LANES>(f2_sum(s1)) * a.inv_d : 0.0f;
      const float m2 = lanes_sum<LANES>(f2_sum(s2)) * a.inv_d;
      // rstd (dn - m1 - n m2)
#pragma unroll
      for (int e = 0; e < E; ++e)
        dy[e] = f2_fma(dy[e], f2_all(rstd), f2_mul(f2_fma(x[e], f2_all(m2), f2_all(m1)), f2_all(-rstd)));
      q.put(dx_at.p, live, dy);
      if constexpr (GATE) q.put(dz_at.p, live, z);
    }
    at.next(a.L);
    dx_at.next(at);
    if constexpr (GATE) dz_at.next(at);
  }
  // the CTA's sums, rows in order; the ring is no longer read, but copies may still be landing
  asm volatile("cp.async.wait_all;\n" ::: "memory");
  __syncthreads();
  float2* sums = reinterpret_cast<float2*>(rings);  // [row of the CTA][channel]
  constexpr int kWide = LANES * NI * V, kRows = kNormThreads / LANES;
  float flat_w[2 * E], flat_b[2 * E];
  Lane::unpack(sw, flat_w);
  Lane::unpack(sb, flat_b);
#pragma unroll
  for (int c = 0; c < NI * V; ++c)
    sums[threadIdx.x / LANES * kWide + (c / V * LANES + q.sub) * V + c % V] =
        make_float2(flat_w[c], flat_b[c]);
  __syncthreads();
  const int keep = a.per_channel ? q.hb : 1;  // sums that stay apart
  for (int i = threadIdx.x; i < keep * a.D; i += kNormThreads) {
    const int j = i / a.D, d = i % a.D;
    if (a.per_channel && q.first_head + j >= a.H) continue;
    float2 s = make_float2(0.0f, 0.0f);
    for (int r = j; r < kRows; r += keep) {
      const float2 v = sums[r * kWide + d];
      s.x += v.x;
      s.y += v.y;
    }
    float* p = a.partials +
               (a.per_channel ? ((int64_t)q.part * a.H + q.first_head + j) : (int64_t)blockIdx.x) * 2 * a.D;
    p[d] = s.x;
    p[a.D + d] = s.y;
  }
}

// ---- heads of more than 1024 channels: one CTA per row ------------------------------------------

// Sums of (p, q) over the CTA, the same in every thread.
__device__ __forceinline__ float2 cta_sum(float p, float q) {
  __shared__ float2 part[kNormThreads / 32];
  p = lanes_sum<32>(p);
  q = lanes_sum<32>(q);
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

template <int NI>
__device__ __forceinline__ float normalise_row(const NormArgs& a, float* x) {
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
  const float rstd = rsqrtf(fmaf(cta_sum(s, 0.0f).x, a.inv_d, a.eps));
#pragma unroll
  for (int i = 0; i < NI; ++i) x[i] *= rstd;
  return rstd;
}

template <typename Act, int NI>
__global__ void __launch_bounds__(kNormThreads) norm_wide_kernel(NormArgs a) {
  const int64_t rows = (int64_t)a.B * a.L * a.H;
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const int h = (int)(r % a.H), l = (int)(r / a.H % a.L), b = (int)(r / a.H / a.L);
    if (l >= seq_len(a.lens, b, a.L)) continue;
    float x[NI], z[NI];
    row_load<Act, NI>(a.x, row_offset(a.x, b, l, h), a.D, x);
    if (a.z.p) row_load<Act, NI>(a.z, row_offset(a.z, b, l, h), a.D, z);
    normalise_row<NI>(a, x);
    const int64_t base = a.per_channel ? (int64_t)h * a.D : 0;
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

// CTA = (part, head): every parts-th token of its head.
template <typename Act, int NI>
__global__ void __launch_bounds__(kNormThreads) norm_wide_backward_kernel(NormArgs a, int parts) {
  let_next_launch();
  const int h = (int)(blockIdx.x % (unsigned)a.H), part = (int)(blockIdx.x / (unsigned)a.H);
  const int64_t base = a.per_channel ? (int64_t)h * a.D : 0;
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
    const float rstd = normalise_row<NI>(a, x);
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
    for (int i = 0; i < NI; ++i) dy[i] = (dy[i] - fmaf(x[i], m2, m1)) * rstd;
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

}  // namespace gdnq
