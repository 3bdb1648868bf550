// Gated scan h_t = a_t h_{t-1} + s(g_t) x_t, a_t = e^{g_t}, and its gradients
// (include/gdnq_layer.h).
//
// Mathematics. A run of up to 16 tokens acts on the state as h -> A h + B, with A = e^{sum g} and B
// its scan from zero, so that runs can be scanned side by side and joined: A is formed from the sum
// of the gates, one rounding for the run, and is a product over several runs. The gradient runs from
// the last token to the first in the same way: with c the gradient that reaches a token's state from
// behind, dh = grad_o + c, and c <- a dh, a run acts as c -> A c + R with the same A.
//
// Split. A warp takes 64 channels and T consecutive tokens at a time in registers; W warps
// of a CTA (a group) and CL CTAs of a cluster take the runs that follow one another, join them
// through shared memory, and walk the sequence together, the next tile's loads under way while
// the present one is scanned. Each array is read and written once, but for few and long sequences,
// whose spans' effects are found by a pass of their own (see SpanLink).
#pragma once

#include "layer_util.cuh"

namespace gdnq {

// A gate's terms for the two channels of a lane.
struct Gate {
  F2 a, s;  // e^g, s(g)
  F2 r;     // 1 / s of GDN_SCALE_SQRT, 0 where s is 0 (backward pass)
};

// e^g and 1 - e^g. Near zero e^g - 1 = g p(g), p of degree 5 through the Chebyshev points of
// [-0.35, 0.35], off by at most 2.6e-8 of itself (half an fp32 step is 6.0e-8), so that neither
// 1 - e^g nor a gate near one loses digits; elsewhere by the hardware's exponential, which takes
// e^g below 2^-126 as zero.
__device__ __forceinline__ void exp_and_rest(F2 g, F2& a, F2& m) {
  F2 p = f2_all(-0.0013934532180428505f);
  p = f2_fma(p, g, f2_all(-0.008369861170649529f));
  p = f2_fma(p, g, f2_all(-0.04166645556688309f));
  p = f2_fma(p, g, f2_all(-0.1666649878025055f));
  p = f2_fma(p, g, f2_all(-0.5f));
  p = f2_fma(p, g, f2_all(-1.0f));
  p = f2_mul(p, g);
  float g0, g1, y0, y1, p0, p1;
  f2_get(g, g0, g1);
  f2_get(f2_mul(g, f2_all(1.4426950408889634f)), y0, y1);
  y0 = exp2_hw(y0);
  y1 = exp2_hw(y1);
  f2_get(p, p0, p1);
  const bool near0 = fabsf(g0) <= 0.35f, near1 = fabsf(g1) <= 0.35f;
  m = f2(near0 ? p0 : 1.0f - y0, near1 ? p1 : 1.0f - y1);
  a = f2(near0 ? 1.0f - p0 : y0, near1 ? 1.0f - p1 : y1);
}

template <int SCALE, bool BACKWARD = false>
__device__ __forceinline__ Gate gate_of(F2 g) {
  Gate q;
  F2 m;
  exp_and_rest(g, q.a, m);
  q.s = f2_all(1.0f);
  q.r = f2_all(0.0f);
  if constexpr (SCALE == GDN_SCALE_COMPLEMENT) q.s = m;
  if constexpr (SCALE == GDN_SCALE_SQRT) {
    const F2 var = f2_mul(m, f2_fma(m, f2_all(-1.0f), f2_all(2.0f)));  // 1 - a^2
    float v0, v1;
    f2_get(var, v0, v1);
    // a variance below the smallest normal number counts as zero
    q.r = f2(rsqrt_hw(fmaxf(v0, 0x1p-126f)), rsqrt_hw(fmaxf(v1, 0x1p-126f)));
    q.s = f2_mul(var, q.r);
    if constexpr (BACKWARD) {
      float r0, r1;
      f2_get(q.r, r0, r1);
      q.r = f2(v0 > 0.0f ? r0 : 0.0f, v1 > 0.0f ? r1 : 0.0f);
    }
  }
  return q;
}

__device__ __forceinline__ F2 run_decay(F2 g_sum) {
  F2 a, m;
  exp_and_rest(g_sum, a, m);
  return a;
}

// The channels of a slab, and a lane's two of them: neighbours (STEP = 1), which are moved as one,
// or 32 apart (STEP = 32), one by one, where the arrays' alignment does not allow that.
constexpr int kScanSlab = 64;

struct ScanLane {
  int c;             // the first one
  bool live, both;   // whether it exists, and the second
  int h, d, h2, d2;  // their places, or that of channel 0, or of the first
};

template <int STEP>
__device__ __forceinline__ ScanLane scan_lane(const ScanArgs& a, int slab) {
  const int lane = threadIdx.x & 31;
  ScanLane l;
  l.c = slab * kScanSlab + (STEP == 1 ? 2 * lane : lane);
  l.live = l.c < a.C;
  l.both = STEP == 1 ? l.live : l.c + STEP < a.C;
  l.h = l.live ? l.c / a.D : 0;
  l.d = l.live ? l.c % a.D : 0;
  l.h2 = l.both ? (l.c + STEP) / a.D : l.h;
  l.d2 = l.both ? (l.c + STEP) % a.D : l.d;
  return l;
}

// The two channels as they lie in memory.
template <typename T, int STEP>
struct Raw {
  T e[2];
  __device__ __forceinline__ F2 get() const { return f2(Num<T>::to_f(e[0]), Num<T>::to_f(e[1])); }
  __device__ __forceinline__ void set(F2 f) {
    float lo, hi;
    f2_get(f, lo, hi);
    e[0] = Num<T>::from_f(lo);
    e[1] = Num<T>::from_f(hi);
  }
};
template <>
struct Raw<float, 1> {
  float2 v;
  __device__ __forceinline__ F2 get() const { return f2(v.x, v.y); }
  __device__ __forceinline__ void set(F2 f) { f2_get(f, v.x, v.y); }
};
template <>
struct Raw<__nv_bfloat16, 1> {
  uint32_t v;
  __device__ __forceinline__ F2 get() const { return f2(bf16_lo(v), bf16_hi(v)); }
  __device__ __forceinline__ void set(F2 f) {
    float lo, hi;
    f2_get(f, lo, hi);
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    v = *reinterpret_cast<const uint32_t*>(&h);
  }
};

// A lane's column of a token array: its channels of every token. Rows are reached by 32-bit
// offsets from the run's first one (the C entry points bound the stride). The stride passes
// through an empty asm statement for every run: the compiler otherwise keeps the offsets of all T
// rows of all arrays in registers through the loop over tiles, and spills.
__device__ __forceinline__ int opaque(int s) {
  asm volatile("" : "+r"(s));
  return s;
}

template <typename T, int STEP>
struct Column {
  T *p, *q;  // the first channel; the second one, or the first where it does not exist
  int sl;
  bool both;
  __device__ __forceinline__ Column(const Tok& t, int b, const ScanLane& l)
      : p(static_cast<T*>(t.p) + channel_offset(t, b, l.h, l.d)),
        q(static_cast<T*>(t.p) + channel_offset(t, b, l.h2, l.d2)), sl((int)t.sl), both(l.both) {}
  struct Run {
    T *p, *q;
    int sl;
    bool both;
    __device__ __forceinline__ Raw<T, STEP> load(int j) const {
      Raw<T, STEP> r;
      r.e[0] = p[j * sl];
      r.e[1] = q[j * sl];
      return r;
    }
    __device__ __forceinline__ void store(int j, F2 f) const {
      Raw<T, STEP> r;
      r.set(f);
      p[j * sl] = r.e[0];
      if (both) q[j * sl] = r.e[1];
    }
  };
  __device__ __forceinline__ Run run(int t) const {
    const int s = opaque(sl);
    return Run{p + (int64_t)t * s, q + (int64_t)t * s, s, both};
  }
};

template <typename T>
struct Column<T, 1> {
  T* p;
  int sl;
  __device__ __forceinline__ Column(const Tok& t, int b, const ScanLane& l)
      : p(static_cast<T*>(t.p) + channel_offset(t, b, l.h, l.d)), sl((int)t.sl) {}
  struct Run {
    T* p;
    int sl;
    __device__ __forceinline__ Raw<T, 1> load(int j) const {
      return *reinterpret_cast<const Raw<T, 1>*>(p + j * sl);
    }
    __device__ __forceinline__ void store(int j, F2 f) const {
      Raw<T, 1> r;
      r.set(f);
      *reinterpret_cast<Raw<T, 1>*>(p + j * sl) = r;
    }
  };
  __device__ __forceinline__ Run run(int t) const {
    const int s = opaque(sl);
    return Run{p + (int64_t)t * s, s};
  }
};

// The lane's two channels of an fp32 state that begins with its first one.
template <int STEP>
__device__ __forceinline__ F2 state_load(const float* p, bool both) {
  return f2(p[0], STEP == 1 || both ? p[STEP] : 0.0f);
}

template <int STEP>
__device__ __forceinline__ void state_store(float* p, bool both, F2 f) {
  float lo, hi;
  f2_get(f, lo, hi);
  p[0] = lo;
  if (STEP == 1 || both) p[STEP] = hi;
}

// The tokens of a warp's runs, tile after tile, as the scans read them: gate, input and (backward)
// the gradient of the output. start() begins with the run at t0, `step` tokens from one tile to
// the next; take() makes the next run readable; next() may begin the loads after it; finish() waits for what is still
// under way.
//
// RunsInRegisters: any alignment, one tile ahead in registers.
template <typename Act, int STEP, int T, bool BACKWARD>
struct RunsInRegisters {
  static constexpr int kStep = STEP, kTokens = T;
  static constexpr int kBytes = 0;  // shared memory per warp
  Column<float, STEP> gate;
  Column<Act, STEP> in, grad;
  bool live;
  int len, t0, step;
  Raw<float, STEP> next_g[T];
  Raw<Act, STEP> next_x[T], next_d[BACKWARD ? T : 1], now_x[T], now_d[BACKWARD ? T : 1];

  __device__ __forceinline__ RunsInRegisters(const ScanArgs& a, uint8_t*, int b, int slab, int len_)
      : gate(a.g, b, scan_lane<STEP>(a, slab)), in(a.x, b, scan_lane<STEP>(a, slab)),
        grad(BACKWARD ? a.grad_o : a.x, b, scan_lane<STEP>(a, slab)),
        live(scan_lane<STEP>(a, slab).live), len(len_) {}
  __device__ __forceinline__ void fetch() {
    const auto rg = gate.run(t0);
    const auto rx = in.run(t0), rd = grad.run(t0);
    const bool whole = live && t0 >= 0 && t0 + T <= len;
#pragma unroll
    for (int j = 0; j < T; ++j) {
      next_g[j] = {};
      next_x[j] = {};
      if constexpr (BACKWARD) next_d[j] = {};
      if (whole || (live && t0 >= 0 && t0 + j < len)) {
        next_g[j] = rg.load(j);
        next_x[j] = rx.load(j);
        if constexpr (BACKWARD) next_d[j] = rd.load(j);
      }
    }
    t0 += step;
  }
  __device__ __forceinline__ void start(int t, int step_) {
    t0 = t;
    step = step_;
    fetch();
  }
  __device__ __forceinline__ void take() {
#pragma unroll
    for (int j = 0; j < T; ++j) {
      now_x[j] = next_x[j];
      if constexpr (BACKWARD) now_d[j] = next_d[j];
    }
  }
  __device__ __forceinline__ void next() { fetch(); }  // once the gates have been read
  __device__ __forceinline__ void finish() {}
  __device__ __forceinline__ F2 g(int j) const { return next_g[j].get(); }
  __device__ __forceinline__ F2 x(int j) const { return now_x[j].get(); }
  __device__ __forceinline__ F2 grad_o(int j) const { return now_d[j].get(); }
};

// RunsInShared: rows that 16-byte pieces cover, copied asynchronously STAGES - 1 tiles ahead into
// a ring of the warp's own (lane l's channels 2 l and 2 l + 1 of the slab's 64, no bank is asked
// twice), so that neither the rows in flight nor their addresses take registers.
template <typename Act, int T, int STAGES, bool BACKWARD>
struct RunsInShared {
  static constexpr int kStep = 1, kTokens = T;
  static constexpr int kWide = kScanSlab;
  static constexpr int kAct = T * kWide * (int)sizeof(Act);
  static constexpr int kStage = T * kWide * 4 + kAct * (BACKWARD ? 2 : 1);
  static constexpr int kBytes = STAGES * kStage;

  // One lane's pieces of one array: `rows` rows by one instruction of the warp.
  template <typename E>
  struct Piece {
    static constexpr int kElems = 16 / (int)sizeof(E), kPieces = kWide / kElems;
    static constexpr int kRows = 32 / kPieces;
    static_assert(T % kRows == 0, "whole instructions per tile");
    const E* p;
    int sl;
    bool live;
    __device__ __forceinline__ Piece(const Tok& t, const ScanArgs& a, int b, int c0) : sl((int)t.sl) {
      const int c = c0 + (threadIdx.x & 31) % kPieces * kElems;
      live = c < a.C;
      p = static_cast<const E*>(t.p) + channel_offset(t, b, live ? c / a.D : 0, live ? c % a.D : 0);
    }
    __device__ __forceinline__ void copy(uint32_t to, int t0, int len) const {
      const int lane = threadIdx.x & 31;
#pragma unroll
      for (int i = 0; i < T; i += kRows) {
        const int t = t0 + i + lane / kPieces;
        const bool ok = live && t >= 0 && t < len;
        const E* from = p + (ok ? (int64_t)t * sl : 0);
        async_piece<16>(to + (uint32_t)((i * kPieces + lane) * 16), from, ok);
      }
    }
  };

  Piece<float> gate;
  Piece<Act> in, grad;
  int len, t0, step, fill, read;
  uint32_t ring;
  const uint8_t* now;

  __device__ __forceinline__ RunsInShared(const ScanArgs& a, uint8_t* shared, int b, int slab, int len_)
      : gate(a.g, a, b, slab * kWide), in(a.x, a, b, slab * kWide),
        grad(BACKWARD ? a.grad_o : a.x, a, b, slab * kWide), len(len_), fill(0), read(0), ring(smem_u32(shared)), now(shared) {}
  __device__ __forceinline__ void fetch() {
    const uint32_t to = ring + (uint32_t)(fill * kStage);
    gate.copy(to, t0, len);
    in.copy(to + T * kWide * 4, t0, len);
    if constexpr (BACKWARD) grad.copy(to + T * kWide * 4 + kAct, t0, len);
    asm volatile("cp.async.commit_group;\n" ::: "memory");
    fill = fill + 1 == STAGES ? 0 : fill + 1;
    t0 += step;
  }
  __device__ __forceinline__ void start(int t, int step_) {
    t0 = t;
    step = step_;
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) fetch();
    now -= kStage;
    read = -1;
  }
  __device__ __forceinline__ void take() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(STAGES - 2) : "memory");
    __syncwarp();  // the other lanes' pieces too, and all have read the tile before
    ++read;
    now += kStage;
    if (read == STAGES) {
      read = 0;
      now -= kBytes;
    }
    fetch();
  }
  __device__ __forceinline__ void next() {}
  __device__ __forceinline__ void finish() { asm volatile("cp.async.wait_all;\n" ::: "memory"); }
  __device__ __forceinline__ F2 g(int j) const {
    return reinterpret_cast<const Raw<float, 1>*>(now)[j * 32 + (threadIdx.x & 31)].get();
  }
  __device__ __forceinline__ F2 x(int j) const {
    return reinterpret_cast<const Raw<Act, 1>*>(now + T * kWide * 4)[j * 32 + (threadIdx.x & 31)].get();
  }
  __device__ __forceinline__ F2 grad_o(int j) const {
    return reinterpret_cast<const Raw<Act, 1>*>(now + T * kWide * 4 + kAct)[j * 32 + (threadIdx.x & 31)].get();
  }
};

// One lane's share of what runs hand each other.
struct Link {
  F2 a, b;
};

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::
                   : "memory");
}

// Stores v at the place that p has in the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ void cluster_store(Link* p, int rank, Link v) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("st.shared::cluster.v2.b64 [%0], {%1, %2};\n" ::"r"(at), "l"(v.a.v), "l"(v.b.v)
               : "memory");
}

constexpr int scan_groups(int W) { return W == 1 ? 8 : 1; }
constexpr int scan_threads(int W) { return 32 * W * scan_groups(W); }

// Few sequences of many tokens: each is split into spans, which CTAs of their own take side by side.
// A first kernel leaves what every span does to the state; a span's state is then what the spans
// before it (backward, behind it) make of the sequence's. It reads a part of the data twice, where
// one chain of clusters would leave most of the machine idle.
//
// The decay of a span, or of many, need not be a number where no state ever meets it: gates a little
// above 1 over a state of zero. So it is also kept with an exponent of its own, a 2^e with 1 <= a < 2
// (or a is 0, infinite or NaN). Below 2^-300 it takes every fp32 state to zero and is zero, above
// 2^300 it takes every other state beyond fp32 and is 2^300. To join spans by such decays is bound by
// their instructions (64 channels x 131072 tokens, 256 spans: 37 us, 33 with plain numbers), so that is
// for sequences with a gate above 1; elsewhere no product of decays is above 1 either.
struct alignas(16) SpanDecay {
  F2 a;
  int e[2];
};
// What a span does: h -> p h + b, with p = a 2^e, or 2 where the span has a gate above 1: then the
// decay is to be taken from there.
struct alignas(16) SpanLink {
  F2 b, p;
};

// Takes the exponent of a (normal, 0, infinite or NaN) into e, which is 0 with a decay of zero.
__device__ __forceinline__ float scaled(float a, int& e) {
  const uint32_t bits = __float_as_uint(a), field = bits >> 23 & 255;
  const int shift = field == 255 ? 0 : (int)field - 127;
  e = min(e + shift, 300);
  const bool zero = field == 0 || e < -300;
  e = zero ? 0 : e;
  return zero ? 0.0f : __uint_as_float(bits - ((uint32_t)shift << 23));
}

__device__ __forceinline__ F2 scaled(F2 a, int (&e)[2]) {
  float lo, hi;
  f2_get(a, lo, hi);
  lo = scaled(lo, e[0]);
  hi = scaled(hi, e[1]);
  return f2(lo, hi);
}

// The part of 2^e within [2^-100, 2^100]; the rest of e stays.
__device__ __forceinline__ float take_power(int& e) {
  const int part = max(-100, min(e, 100));
  e -= part;
  return __uint_as_float((uint32_t)(part + 127) << 23);
}

__device__ __forceinline__ F2 take_power(int (&e)[2]) {
  const float lo = take_power(e[0]), hi = take_power(e[1]);
  return f2(lo, hi);
}

// The factors of a 2^e, e within +-300, one after the other.
__device__ __forceinline__ void factors(const SpanDecay& d, F2 (&f)[3]) {
  int e[2] = {d.e[0], d.e[1]};
  f[0] = f2_mul(take_power(e), d.a);
  f[1] = take_power(e);
  f[2] = take_power(e);
}

__device__ __forceinline__ F2 decayed(const F2 (&f)[3], F2 h, F2 b) {
  return f2_fma(f2_mul(f2_mul(h, f[0]), f[1]), f[2], b);
}

__device__ __forceinline__ bool above(F2 f, float limit) {
  float lo, hi;
  f2_get(f, lo, hi);
  return lo > limit || hi > limit;
}

// The workspace: links [link][unit][32], link 0 of a unit its first state (backward the gradient of
// its last one), link i + 1 span i's; behind them the spans' decays in the same order.
__device__ __forceinline__ SpanLink* span_links(const ScanArgs& a, int64_t units, int64_t unit, int link) {
  return static_cast<SpanLink*>(a.spans) + (link * units + unit) * 32 + (threadIdx.x & 31);
}

__device__ __forceinline__ SpanDecay* span_decays(const ScanArgs& a, int64_t units, int64_t unit, int link) {
  return reinterpret_cast<SpanDecay*>(span_links(a, units, unit, a.spans_per_unit + 1 + link));
}

// A warp's part of a sequence: its b and the factors of its decay, [4][W][32] in shared memory.
template <int W>
struct SpanPart {
  static __device__ __forceinline__ void put(F2* shared, F2 b, const F2 (&f)[3]) {
    shared[threadIdx.x] = b;
#pragma unroll
    for (int k = 0; k < 3; ++k) shared[(k + 1) * W * 32 + threadIdx.x] = f[k];
  }
  static __device__ __forceinline__ F2 apply(const F2* shared, int w, F2 h) {
    const F2* at = shared + w * 32 + (threadIdx.x & 31);
    const F2 f[3] = {at[W * 32], at[2 * W * 32], at[3 * W * 32]};
    return decayed(f, h, at[0]);
  }
};

// What the links from `from` on, `count` of them in steps of `step`, make of the state: an equal part
// of them joined by each of the CTA's W warps, the parts in shared memory. The same in every warp.
template <int W>
__device__ __forceinline__ F2 join_spans(const ScanArgs& a, int64_t units, int64_t unit, F2 state,
                                         int from, int count, int step, F2* shared) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int share = (count + W - 1) / W, begin = w * share, end = min(begin + share, count);
  SpanLink all = {f2_all(0.0f), f2_all(1.0f)};
  bool grows = false;
#pragma unroll 8
  for (int i = begin; i < end; ++i) {
    const SpanLink l = *span_links(a, units, unit, from + i * step);
    grows = grows || above(l.p, 1.0f);
    all.b = f2_fma(l.p, all.b, l.b);
    all.p = f2_mul(l.p, all.p);
  }
  F2 f[3] = {all.p, f2_all(1.0f), f2_all(1.0f)};
  if (__syncthreads_or(grows)) {
    SpanDecay d = {f2_all(1.0f), {0, 0}};
    all.b = f2_all(0.0f);
    for (int i = begin; i < end; ++i) {
      const SpanDecay next = *span_decays(a, units, unit, from + i * step);
      factors(next, f);
      all.b = decayed(f, all.b, span_links(a, units, unit, from + i * step)->b);
      d.e[0] += next.e[0];
      d.e[1] += next.e[1];
      d.a = scaled(f2_mul(next.a, d.a), d.e);
    }
    factors(d, f);
  }
  SpanPart<W>::put(shared, all.b, f);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < W; ++i) state = SpanPart<W>::apply(shared, i, state);
  __syncthreads();
  return state;
}

// A warp takes an eighth of a span. Backward `in` is grad_o, and a run acts on the gradient that
// comes from behind.
template <typename Act, int SCALE, class Runs, bool BACKWARD>
__global__ void __launch_bounds__(256, 2) scan_span_kernel(ScanArgs a, int slabs) {
  constexpr int W = 8, T = Runs::kTokens;
  extern __shared__ __align__(128) uint8_t rings[];
  __shared__ F2 part[4 * W * 32];
  __shared__ SpanDecay decay[W][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t units = (int64_t)a.B * slabs, unit = blockIdx.x % units;
  const int span = (int)(blockIdx.x / units);
  const int b = (int)(unit / slabs), slab = (int)(unit % slabs);
  const int len = seq_len(a.lens, b, a.L), first = span * a.span_tokens;
  if (span == 0 && w == 0) {
    // the state before the sequence (the gradient behind it): the second kernel's CTAs read it here,
    // since hT may be h0 (grad_h0 grad_hT)
    const ScanLane me = scan_lane<Runs::kStep>(a, slab);
    const int64_t state = (int64_t)b * a.C + me.c;
    span_links(a, units, unit, 0)->b =
        a.h0 && me.live ? state_load<Runs::kStep>(a.h0 + state, me.both) : f2_all(0.0f);
  }
  if (first >= len) return;
  const int share = a.span_tokens / W, begin = first + w * share, end = min(begin + share, len);
  Runs runs(a, rings + w * Runs::kBytes, b, slab, end);
  const int tiles = end > begin ? (end - begin + T - 1) / T : 0;
  runs.start(BACKWARD ? begin + (tiles - 1) * T : begin, BACKWARD ? -T : T);
  F2 state = f2_all(0.0f);
  SpanDecay all = {f2_all(1.0f), {0, 0}};
  float most = 0.0f;  // of the gates' logs
  for (int tile = 0; tile < tiles; ++tile) {
    runs.take();
    F2 g_sum = f2_all(0.0f), at[T];
#pragma unroll
    for (int j = 0; j < T; ++j) {
      const F2 gj = runs.g(j);
      const Gate q = gate_of<BACKWARD ? GDN_SCALE_NONE : SCALE>(gj);
      float g0, g1;
      f2_get(gj, g0, g1);
      most = fmaxf(most, fmaxf(g0, g1));
      at[j] = q.a;
      g_sum = f2_add(g_sum, gj);
      if constexpr (!BACKWARD) state = f2_fma(q.a, state, f2_mul(q.s, runs.x(j)));
    }
    if constexpr (BACKWARD) {
#pragma unroll
      for (int j = T - 1; j >= 0; --j) state = f2_mul(at[j], f2_add(runs.x(j), state));
    }
    all.a = f2_mul(all.a, run_decay(g_sum));
    // 128 tokens multiply by less than e^88 < 2^127
    if (tile % (128 / T) == 128 / T - 1) all.a = scaled(all.a, all.e);
    runs.next();
  }
  runs.finish();
  all.a = scaled(all.a, all.e);
  F2 f[3];
  factors(all, f);
  SpanPart<W>::put(part, state, f);
  decay[w][lane] = all;
  const bool grows = __syncthreads_or(most > 0.0f);
  if (w == 0) {
    state = f2_all(0.0f);
#pragma unroll
    for (int i = 0; i < W; ++i) state = SpanPart<W>::apply(part, BACKWARD ? W - 1 - i : i, state);
#pragma unroll
    for (int i = 1; i < W; ++i) {
      all.a = f2_mul(all.a, decay[i][lane].a);  // of eight numbers below 2
      all.e[0] += decay[i][lane].e[0];
      all.e[1] += decay[i][lane].e[1];
    }
    all.a = scaled(all.a, all.e);
    factors(all, f);
    *span_links(a, units, unit, span + 1) =
        SpanLink{state, grows ? f2_all(2.0f) : decayed(f, f2_all(1.0f), f2_all(0.0f))};
    *span_decays(a, units, unit, span + 1) = all;
  }
}

// The joins' two buffers of links, which hold the W parts of a sequence before the first tile.
template <int W>
__device__ __forceinline__ F2* parts_of(Link (&agg)[2][W][32]) {
  static_assert(sizeof(agg) == 4 * W * 32 * sizeof(F2), "as large");
  return &agg[0][0][0].a;
}

template <typename Act, int SCALE, class Runs, int W, int CL, int MINB, bool SPLIT = false>
__global__ void __launch_bounds__(scan_threads(W), MINB) scan_kernel(ScanArgs a, int slabs) {
  static_assert(!SPLIT || (CL == 1 && W > 1), "a span is one CTA's");
  constexpr int kGroups = scan_groups(W), STEP = Runs::kStep, T = Runs::kTokens;
  extern __shared__ __align__(128) uint8_t rings[];
  static_assert(GDN_SCAN_CHUNK % T == 0, "kept states stand where runs begin");
  __shared__ alignas(16) Link agg[W > 1 ? 2 : 1][W][W > 1 ? 32 : 1];
  __shared__ alignas(16) Link across[CL > 1 ? 2 : 1][CL][CL > 1 ? 32 : 1];
  const int lane = threadIdx.x & 31, w = W > 1 ? threadIdx.x >> 5 : 0;
  const int rank = CL > 1 ? (int)(blockIdx.x % CL) : 0;
  const int64_t units = SPLIT ? (int64_t)a.B * slabs : 0;
  const int span = SPLIT ? (int)(blockIdx.x / units) : 0;
  const int64_t unit = SPLIT ? blockIdx.x % units
                       : CL > 1 ? blockIdx.x / CL
                                : (int64_t)blockIdx.x * kGroups + (W > 1 ? 0 : threadIdx.x >> 5);
  if (W == 1 && unit >= (int64_t)a.B * slabs) return;  // no barrier waits for this warp
  const int b = (int)(unit / slabs), slab = (int)(unit % slabs);
  const ScanLane me = scan_lane<STEP>(a, slab);
  const bool live = me.live;
  const int length = seq_len(a.lens, b, a.L);
  const int first = SPLIT ? span * a.span_tokens : 0;
  if (SPLIT && span > 0 && first >= length) return;
  const int len = SPLIT ? min(length, first + a.span_tokens) : length;  // this CTA's end
  const Column<Act, STEP> o(a.o, b, me);
  Runs runs(a, rings + (threadIdx.x >> 5) * Runs::kBytes, b, slab, len);
  const int64_t state = (int64_t)b * a.C + me.c;
  float* hist = a.hist && live
                    ? a.hist + (int64_t)b * ((a.L + GDN_SCAN_CHUNK - 1) / GDN_SCAN_CHUNK) * a.C + me.c
                    : nullptr;
  F2 carry;  // before the tile
  if constexpr (SPLIT)
    carry = join_spans<W>(a, units, unit, span_links(a, units, unit, 0)->b, 1, span, 1, parts_of(agg));
  else
    carry = a.h0 && live ? state_load<STEP>(a.h0 + state, me.both) : f2_all(0.0f);

  constexpr int kTile = CL * W * T;
  int t0 = first + (rank * W + w) * T;
  runs.start(t0, kTile);
  if constexpr (CL > 1) cluster_barrier();  // every CTA of the cluster runs before it is written to
  int buf = 0;
  for (int tile = first; tile < len; tile += kTile, t0 += kTile, buf ^= 1) {
    runs.take();
    F2 at[T], u[T], g_sum = f2_all(0.0f), local = f2_all(0.0f);
#pragma unroll
    for (int j = 0; j < T; ++j) {
      const F2 gj = runs.g(j);
      const Gate q = gate_of<SCALE>(gj);
      at[j] = q.a;
      u[j] = SCALE == GDN_SCALE_NONE ? runs.x(j) : f2_mul(q.s, runs.x(j));
      if constexpr (W > 1) {
        g_sum = f2_add(g_sum, gj);
        local = f2_fma(q.a, local, u[j]);
      }
    }
    runs.next();
    F2 h = carry;  // the state before the warp's run
    if constexpr (W > 1) {
      agg[buf][w][lane] = Link{run_decay(g_sum), local};
      __syncthreads();
      if constexpr (CL > 1) {
        // the CTA's run, and the part of it before this warp's
        Link before = {f2_all(1.0f), f2_all(0.0f)}, all = before;
#pragma unroll
        for (int i = 0; i < W; ++i) {
          if (i == w) before = all;
          const Link l = agg[buf][i][lane];
          all.a = f2_mul(l.a, all.a);
          all.b = f2_fma(l.a, all.b, l.b);
        }
        for (int r = w; r < CL; r += W) cluster_store(&across[buf][rank][lane], r, all);
        cluster_barrier();
#pragma unroll
        for (int i = 0; i < CL; ++i) {
          if (i == rank) h = f2_fma(before.a, carry, before.b);
          const Link l = across[buf][i][lane];
          carry = f2_fma(l.a, carry, l.b);
        }
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i) {
          if (i == w) h = carry;
          const Link l = agg[buf][i][lane];
          carry = f2_fma(l.a, carry, l.b);
        }
      }
    }
    if (hist && t0 % GDN_SCAN_CHUNK == 0 && t0 < len)
      state_store<STEP>(hist + (int64_t)(t0 / GDN_SCAN_CHUNK) * a.C, me.both, h);
    const auto ro = o.run(t0);
    if (live && t0 + T <= len) {
#pragma unroll
      for (int j = 0; j < T; ++j) {
        h = f2_fma(at[j], h, u[j]);
        ro.store(j, h);
      }
    } else {
#pragma unroll
      for (int j = 0; j < T; ++j) {
        h = f2_fma(at[j], h, u[j]);
        if (live && t0 + j < len) ro.store(j, h);
      }
    }
    if constexpr (W == 1) carry = h;
  }
  runs.finish();  // copies behind the last tile
  if (a.hT && live && rank == 0 && w == 0 && len == length) state_store<STEP>(a.hT + state, me.both, carry);
}

// A CTA's tile is one chunk between kept states; with one warp a unit (sequences of one run) eight
// units share a CTA.
template <typename Act, int SCALE, class Runs, int W, int CL, int MINB, bool SPLIT = false>
__global__ void __launch_bounds__(scan_threads(W), MINB) scan_backward_kernel(ScanArgs a, int slabs) {
  constexpr int T = Runs::kTokens, STEP = Runs::kStep, kGroups = scan_groups(W);
  static_assert(W * T == GDN_SCAN_CHUNK || (W == 1 && CL == 1), "tiles begin at kept states");
  extern __shared__ __align__(128) uint8_t rings[];
  __shared__ alignas(16) Link agg[W > 1 ? 2 : 1][W][W > 1 ? 32 : 1];  // decay and scan of each run
  __shared__ F2 agg_back[W > 1 ? 2 : 1][W][W > 1 ? 32 : 1];           // its scan of the gradient
  __shared__ alignas(16) Link across[CL > 1 ? 2 : 1][CL][CL > 1 ? 32 : 1];
  const int lane = threadIdx.x & 31, w = W > 1 ? threadIdx.x >> 5 : 0;
  const int rank = CL > 1 ? (int)(blockIdx.x % CL) : 0;
  const int64_t units = SPLIT ? (int64_t)a.B * slabs : 0;
  const int span = SPLIT ? (int)(blockIdx.x / units) : 0;
  const int64_t unit = SPLIT ? blockIdx.x % units
                       : CL > 1 ? blockIdx.x / CL
                                : (int64_t)blockIdx.x * kGroups + (W > 1 ? 0 : threadIdx.x >> 5);
  if (W == 1 && unit >= (int64_t)a.B * slabs) return;  // no barrier waits for this warp
  const int b = (int)(unit / slabs), slab = (int)(unit % slabs);
  const ScanLane me = scan_lane<STEP>(a, slab);
  const bool live = me.live;
  const int length = seq_len(a.lens, b, a.L);
  const int begin = SPLIT ? span * a.span_tokens : 0;
  if (SPLIT && span > 0 && begin >= length) return;
  const int len = SPLIT ? min(length, begin + a.span_tokens) : length;  // this CTA's end
  const Column<Act, STEP> gx(a.grad_x, b, me);
  const Column<float, STEP> gg(a.grad_g, b, me);
  Runs runs(a, rings + (threadIdx.x >> 5) * Runs::kBytes, b, slab, len);
  const int64_t state = (int64_t)b * a.C + me.c;
  const float* hist =
      a.hist + (int64_t)b * ((a.L + GDN_SCAN_CHUNK - 1) / GDN_SCAN_CHUNK) * a.C + me.c;
  // the gradient that reaches the tile's last state from behind
  F2 carry;
  if constexpr (SPLIT) {
    const int last = (length + a.span_tokens - 1) / a.span_tokens;  // the last span's link
    carry = join_spans<W>(a, units, unit, span_links(a, units, unit, 0)->b, last, max(last - span - 1, 0),
                          -1, parts_of(agg));
  } else {
    carry = a.h0 && live ? state_load<STEP>(a.h0 + state, me.both) : f2_all(0.0f);
  }

  // the kept state before the CTA's tile that begins at `first`
  auto kept = [&](int first) {
    return live && first >= begin && first < len
               ? state_load<STEP>(hist + (int64_t)(first / GDN_SCAN_CHUNK) * a.C, me.both)
               : f2_all(0.0f);
  };

  constexpr int kTile = CL * W * T;
  const int tiles = (len - begin + kTile - 1) / kTile;
  int t0 = begin + (tiles - 1) * kTile + (rank * W + w) * T;
  runs.start(t0, -kTile);
  F2 next_h = kept(t0 - w * T);
  if constexpr (CL > 1) cluster_barrier();  // every CTA of the cluster runs before it is written to
  int buf = 0;
  for (int tile = tiles - 1; tile >= 0; --tile, t0 -= kTile, buf ^= 1) {
    runs.take();
    F2 at[T], s[T], r[T], g_sum = f2_all(0.0f), fwd = g_sum, bwd = g_sum, h = next_h;
#pragma unroll
    for (int j = 0; j < T; ++j) {
      const F2 gj = runs.g(j);
      const Gate q = gate_of<SCALE, true>(gj);
      at[j] = q.a;
      s[j] = q.s;
      r[j] = q.r;
      g_sum = f2_add(g_sum, gj);
      fwd = f2_fma(q.a, fwd, f2_mul(q.s, runs.x(j)));
    }
#pragma unroll
    for (int j = T - 1; j >= 0; --j) bwd = f2_mul(at[j], f2_add(runs.grad_o(j), bwd));
    runs.next();
    next_h = kept(t0 - w * T - kTile);
    F2 dc = carry;  // the gradient that reaches the warp's last state from behind
    if constexpr (W > 1) {
      agg[buf][w][lane] = Link{run_decay(g_sum), fwd};
      agg_back[buf][w][lane] = bwd;
      __syncthreads();
      if constexpr (CL > 1) {
        // the CTA's run, and the part of it behind this warp's
        Link behind = {f2_all(1.0f), f2_all(0.0f)}, all = behind;
#pragma unroll
        for (int i = W - 1; i >= 0; --i) {
          if (i == w) behind = all;
          const F2 ai = agg[buf][i][lane].a;
          all.a = f2_mul(ai, all.a);
          all.b = f2_fma(ai, all.b, agg_back[buf][i][lane]);
        }
        for (int r = w; r < CL; r += W) cluster_store(&across[buf][rank][lane], r, all);
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
          const Link l = agg[buf][i][lane];
          if (i < w) h = f2_fma(l.a, h, l.b);
        }
        cluster_barrier();
#pragma unroll
        for (int i = CL - 1; i >= 0; --i) {
          if (i == rank) dc = f2_fma(behind.a, carry, behind.b);
          const Link l = across[buf][i][lane];
          carry = f2_fma(l.a, carry, l.b);
        }
      } else {
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
          const Link l = agg[buf][i][lane];
          if (i < w) h = f2_fma(l.a, h, l.b);
        }
#pragma unroll
        for (int i = W - 1; i >= 0; --i) {
          if (i == w) dc = carry;
          carry = f2_fma(agg[buf][i][lane].a, carry, agg_back[buf][i][lane]);
        }
      }
    }
    F2 before[T];  // the state before each token, and what the slope of s adds to it
#pragma unroll
    for (int j = 0; j < T; ++j) {
      const F2 xj = runs.x(j);
      // with s' = -a for 1 - a and -a^2 / s for sqrt(1 - a^2), grad_g = a dh (h + s' x / a)
      before[j] = h;
      if constexpr (SCALE == GDN_SCALE_COMPLEMENT) before[j] = f2_fma(xj, f2_all(-1.0f), h);
      if constexpr (SCALE == GDN_SCALE_SQRT)
        before[j] = f2_fma(f2_mul(f2_mul(at[j], f2_all(-1.0f)), r[j]), xj, h);
      h = f2_fma(at[j], h, f2_mul(s[j], xj));
    }
    const auto wx = gx.run(t0);
    const auto wg = gg.run(t0);
    const bool whole = live && t0 + T <= len;
#pragma unroll
    for (int j = T - 1; j >= 0; --j) {
      const F2 dh = f2_add(runs.grad_o(j), dc);
      const F2 dx = f2_mul(s[j], dh);
      dc = f2_mul(at[j], dh);
      if (whole || (live && t0 + j < len)) {
        wx.store(j, dx);
        wg.store(j, f2_mul(dc, before[j]));
      }
    }
    if constexpr (W == 1) carry = dc;
  }
  runs.finish();  // copies behind the last tile
  if (a.hT && live && rank == 0 && w == 0 && span == 0) state_store<STEP>(a.hT + state, me.both, carry);
}

}  // namespace gdnq
