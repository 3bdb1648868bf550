// Gated scan h_t = a_t h_{t-1} + s(g_t) x_t, a_t = e^{g_t}, and its gradients
// (include/gdnq_layer.h).
//
// Mathematics. A run of tokens acts on the state as h -> A h + B, with A = e^{sum g} and B its
// scan from zero, so that runs can be scanned side by side and joined: A is formed from the sum
// of the gates, one rounding however long the run. The gradient runs from the last token to the
// first in the same way: with c the gradient that reaches a token's state from behind,
// dh = grad_o + c, and c <- a dh, a run acts as c -> A c + R with the same A.
//
// Split. A warp takes 32 VEC channels and T consecutive tokens at a time in registers; W warps
// of a CTA (a group) and CL CTAs of a cluster take the runs that follow one another, join them
// through shared memory, and walk the sequence together, the next tile's loads under way while
// the present one is scanned. Each array is read and written once.
#pragma once

#include "layer_util.cuh"

namespace gdnq {

constexpr int kScanWarps = 8;  // of a CTA: kScanWarps / W groups, each with a slab of its own

struct Gate {
  float a, s;  // e^g, s(g)
  float r;     // what the slope takes: 1 / s of GDN_SCALE_SQRT
};

// e^g - 1 and e^g. Near zero e^g - 1 = g p(g), p of degree 5 through the Chebyshev points of
// [-0.35, 0.35], off by at most 2.6e-8 of itself (half an fp32 step is 6.0e-8), so that neither
// 1 - e^g nor a gate near one loses digits; elsewhere by the hardware's exponential.
__device__ __forceinline__ void exp_and_m1(float g, float& a, float& e) {
  float p = 0.0013934532180428505f;
  p = fmaf(p, g, 0.008369861170649529f);
  p = fmaf(p, g, 0.04166645556688309f);
  p = fmaf(p, g, 0.1666649878025055f);
  p = fmaf(p, g, 0.5f);
  p = fmaf(p, g, 1.0f);
  const float big = fast_exp(g);
  const bool near = fabsf(g) <= 0.35f;
  e = near ? p * g : big - 1.0f;
  a = near ? 1.0f + e : big;
}

template <int SCALE>
__device__ __forceinline__ Gate gate_of(float g) {
  Gate q;
  float e;
  exp_and_m1(g, q.a, e);
  q.s = 1.0f;
  q.r = 0.0f;
  if constexpr (SCALE == GDN_SCALE_COMPLEMENT) q.s = -e;
  if constexpr (SCALE == GDN_SCALE_SQRT) {
    const float v = -e * (2.0f + e);  // 1 - a^2
    q.r = v == 0.0f ? 0.0f : rsqrtf(v);
    q.s = v * q.r;
  }
  return q;
}

__device__ __forceinline__ float run_decay(float g_sum) {
  float a, e;
  exp_and_m1(g_sum, a, e);
  return a;
}

// VEC consecutive elements as they lie in memory.
template <typename T, int VEC>
struct Raw;
template <>
struct Raw<float, 1> {
  float v;
  __device__ __forceinline__ void get(float* f) const { f[0] = v; }
  __device__ __forceinline__ void set(const float* f) { v = f[0]; }
};
template <>
struct Raw<float, 2> {
  float2 v;
  __device__ __forceinline__ void get(float* f) const { f[0] = v.x, f[1] = v.y; }
  __device__ __forceinline__ void set(const float* f) { v = make_float2(f[0], f[1]); }
};
template <>
struct Raw<__nv_bfloat16, 1> {
  uint16_t v;
  __device__ __forceinline__ void get(float* f) const { f[0] = __uint_as_float((uint32_t)v << 16); }
  __device__ __forceinline__ void set(const float* f) { v = __bfloat16_as_ushort(__float2bfloat16_rn(f[0])); }
};
template <>
struct Raw<__nv_bfloat16, 2> {
  uint32_t v;
  __device__ __forceinline__ void get(float* f) const { f[0] = bf16_lo(v), f[1] = bf16_hi(v); }
  __device__ __forceinline__ void set(const float* f) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[0], f[1]);
    v = *reinterpret_cast<const uint32_t*>(&h);
  }
};

// A lane's column of a token array: VEC channels from flat channel c.
template <typename T, int VEC>
struct Column {
  T* p;
  int64_t sl;
  __device__ __forceinline__ Column(const Tok& t, int b, int h, int d)
      : p(static_cast<T*>(t.p) + channel_offset(t, b, h, d)), sl(t.sl) {}
  // A cursor on the row of token t. The stride passes through an empty asm statement in every
  // tile: the compiler otherwise keeps the offsets of all T rows of all arrays in registers
  // through the loop over tiles, and spills (208 bytes a thread at T = 8, VEC = 2).
  struct Row {
    T* p;
    int64_t sl;
    __device__ __forceinline__ Raw<T, VEC> load() const {
      return *reinterpret_cast<const Raw<T, VEC>*>(p);
    }
    __device__ __forceinline__ void store(const float* f) const {
      Raw<T, VEC> r;
      r.set(f);
      *reinterpret_cast<Raw<T, VEC>*>(p) = r;
    }
    __device__ __forceinline__ void next() { p += sl; }
    __device__ __forceinline__ void prev() { p -= sl; }
  };
  __device__ __forceinline__ Row row(int t) const {
    int64_t s = sl;
    asm volatile("" : "+l"(s));
    return Row{p + t * s, s};
  }
};

// Barrier of the W warps of one group.
template <int W>
__device__ __forceinline__ void group_sync(int group) {
  if constexpr (W == kScanWarps)
    __syncthreads();
  else if constexpr (W > 1)
    asm volatile("bar.sync %0, %1;\n" ::"r"(group + 1), "n"(W * 32) : "memory");
}

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::
                   : "memory");
}

// Stores v at the address that p has in the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ void cluster_store(float* p, int rank, float v) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;\n" ::"r"(at), "f"(v) : "memory");
}

template <typename Act, int SCALE, int VEC, int W, int T, int CL>
__global__ void __launch_bounds__(kScanWarps * 32, 3) scan_kernel(ScanArgs a, int slabs) {
  static_assert(CL == 1 || W == kScanWarps, "a cluster's CTAs have one group each");
  static_assert(GDN_SCAN_CHUNK % T == 0, "kept states stand where runs begin");
  constexpr int kGroups = kScanWarps / W;
  __shared__ float agg[W > 1 ? 2 : 1][kGroups][W > 1 ? W : 1][2 * VEC][W > 1 ? 32 : 1];
  __shared__ float across[CL > 1 ? 2 : 1][CL][2 * VEC][CL > 1 ? 32 : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = warp / W, w = warp % W;
  const int rank = CL > 1 ? (int)(blockIdx.x % CL) : 0;
  const int64_t unit = CL > 1 ? blockIdx.x / CL : (int64_t)blockIdx.x * kGroups + group;
  if (unit >= (int64_t)a.B * slabs) return;  // a whole group (CL == 1: no cluster waits for it)
  const int b = (int)(unit / slabs), c = (int)(unit % slabs) * 32 * VEC + lane * VEC;
  const bool live = c < a.C;
  const int hd = live ? c / a.D : 0, d = live ? c % a.D : 0;
  const int len = seq_len(a.lens, b, a.L);
  const Column<Act, VEC> x(a.x, b, hd, d);
  const Column<float, VEC> g(a.g, b, hd, d);
  const Column<Act, VEC> o(a.o, b, hd, d);
  const int64_t state = (int64_t)b * a.C + c;
  float* hist = a.hist && live
                    ? a.hist + (int64_t)b * ((a.L + GDN_SCAN_CHUNK - 1) / GDN_SCAN_CHUNK) * a.C + c
                    : nullptr;

  float carry[VEC];  // the state before the tile
#pragma unroll
  for (int v = 0; v < VEC; ++v) carry[v] = a.h0 && live ? a.h0[state + v] : 0.0f;

  Raw<float, VEC> next_g[T];
  Raw<Act, VEC> next_x[T];
  auto load = [&](int t0) {
    auto rg = g.row(t0);
    auto rx = x.row(t0);
#pragma unroll
    for (int j = 0; j < T; ++j, rg.next(), rx.next()) {
      next_g[j] = {};
      next_x[j] = {};
      if (live && t0 + j < len) {
        next_g[j] = rg.load();
        next_x[j] = rx.load();
      }
    }
  };

  constexpr int kTile = CL * W * T;
  int t0 = (rank * W + w) * T;
  load(t0);
  if constexpr (CL > 1) cluster_barrier();  // every CTA of the cluster runs before it is written to
  int buf = 0;
  for (int tile = 0; tile < len; tile += kTile, t0 += kTile, buf ^= 1) {
    float at[T][VEC], u[T][VEC], gsum[VEC], local[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) gsum[v] = local[v] = 0.0f;
#pragma unroll
    for (int j = 0; j < T; ++j) {
      float gv[VEC], xv[VEC];
      next_g[j].get(gv);
      next_x[j].get(xv);
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const Gate q = gate_of<SCALE>(gv[v]);
        at[j][v] = q.a;
        u[j][v] = q.s * xv[v];
        gsum[v] += gv[v];
        local[v] = fmaf(at[j][v], local[v], u[j][v]);
      }
    }
    load(t0 + kTile);
    float h[VEC];  // the state before the warp's run
    if constexpr (W == 1) {
#pragma unroll
      for (int v = 0; v < VEC; ++v) h[v] = carry[v];
    } else {
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        agg[buf][group][w][v][lane] = run_decay(gsum[v]);
        agg[buf][group][w][VEC + v][lane] = local[v];
      }
      group_sync<W>(group);
      if constexpr (CL > 1) {
        // the CTA's run, and the part of it before this warp's
        float pa[VEC], pb[VEC], ca[VEC], cb[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          ca[v] = 1.0f;
          cb[v] = 0.0f;
#pragma unroll
          for (int i = 0; i < W; ++i) {
            if (i == w) pa[v] = ca[v], pb[v] = cb[v];
            const float ai = agg[buf][group][i][v][lane];
            ca[v] *= ai;
            cb[v] = fmaf(ai, cb[v], agg[buf][group][i][VEC + v][lane]);
          }
          if (w < CL) {
            cluster_store(&across[buf][rank][v][lane], w, ca[v]);
            cluster_store(&across[buf][rank][VEC + v][lane], w, cb[v]);
          }
        }
        cluster_barrier();
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
#pragma unroll
          for (int i = 0; i < CL; ++i) {
            if (i == rank) h[v] = fmaf(pa[v], carry[v], pb[v]);
            carry[v] = fmaf(across[buf][i][v][lane], carry[v], across[buf][i][VEC + v][lane]);
          }
        }
      } else {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
#pragma unroll
          for (int i = 0; i < W; ++i) {
            if (i == w) h[v] = carry[v];
            carry[v] = fmaf(agg[buf][group][i][v][lane], carry[v],
                            agg[buf][group][i][VEC + v][lane]);
          }
        }
      }
    }
    if (hist && t0 % GDN_SCAN_CHUNK == 0 && t0 < len) {
#pragma unroll
      for (int v = 0; v < VEC; ++v) hist[(int64_t)(t0 / GDN_SCAN_CHUNK) * a.C + v] = h[v];
    }
    auto ro = o.row(t0);
#pragma unroll
    for (int j = 0; j < T; ++j, ro.next()) {
#pragma unroll
      for (int v = 0; v < VEC; ++v) h[v] = fmaf(at[j][v], h[v], u[j][v]);
      if (live && t0 + j < len) ro.store(h);
    }
    if constexpr (W == 1) {
#pragma unroll
      for (int v = 0; v < VEC; ++v) carry[v] = h[v];
    }
  }
  if (a.hT && live && rank == 0 && w == 0) {
#pragma unroll
    for (int v = 0; v < VEC; ++v) a.hT[state + v] = carry[v];
  }
}

template <typename Act, int SCALE, int VEC, int W, int T, int CL>
__global__ void __launch_bounds__(kScanWarps * 32, 2) scan_backward_kernel(ScanArgs a, int slabs) {
  static_assert(W == kScanWarps && W * T == GDN_SCAN_CHUNK, "a CTA's tile is one kept chunk");
  __shared__ float agg[2][W][3 * VEC][32];
  __shared__ float across[CL > 1 ? 2 : 1][CL][2 * VEC][CL > 1 ? 32 : 1];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int rank = CL > 1 ? (int)(blockIdx.x % CL) : 0;
  const int64_t unit = blockIdx.x / CL;
  const int b = (int)(unit / slabs), c = (int)(unit % slabs) * 32 * VEC + lane * VEC;
  const bool live = c < a.C;
  const int hd = live ? c / a.D : 0, d = live ? c % a.D : 0;
  const int len = seq_len(a.lens, b, a.L);
  const Column<Act, VEC> x(a.x, b, hd, d), go(a.grad_o, b, hd, d);
  const Column<float, VEC> g(a.g, b, hd, d);
  const Column<Act, VEC> gx(a.grad_x, b, hd, d);
  const Column<float, VEC> gg(a.grad_g, b, hd, d);
  const int64_t state = (int64_t)b * a.C + c;
  const float* hist =
      a.hist + (int64_t)b * ((a.L + GDN_SCAN_CHUNK - 1) / GDN_SCAN_CHUNK) * a.C + c;

  float carry[VEC];  // the gradient that reaches the tile's last state from behind
#pragma unroll
  for (int v = 0; v < VEC; ++v) carry[v] = a.h0 && live ? a.h0[state + v] : 0.0f;

  Raw<float, VEC> next_g[T];
  Raw<Act, VEC> next_x[T], next_o[T];
  float next_h[VEC];  // the kept state before the CTA's tile
  auto load = [&](int t0) {
    auto rg = g.row(t0);
    auto rx = x.row(t0), rd = go.row(t0);
#pragma unroll
    for (int j = 0; j < T; ++j, rg.next(), rx.next(), rd.next()) {
      next_g[j] = {};
      next_x[j] = {};
      next_o[j] = {};
      if (live && t0 >= 0 && t0 + j < len) {
        next_g[j] = rg.load();
        next_x[j] = rx.load();
        next_o[j] = rd.load();
      }
    }
    const int at = t0 - w * T;
#pragma unroll
    for (int v = 0; v < VEC; ++v)
      next_h[v] = live && at >= 0 && at < len ? hist[(int64_t)(at / GDN_SCAN_CHUNK) * a.C + v] : 0.0f;
  };

  constexpr int kTile = CL * GDN_SCAN_CHUNK;
  const int tiles = (int)(((int64_t)len + kTile - 1) / kTile);
  int t0 = (tiles - 1) * kTile + rank * GDN_SCAN_CHUNK + w * T;
  load(t0);
  if constexpr (CL > 1) cluster_barrier();  // every CTA of the cluster runs before it is written to
  int buf = 0;
  for (int tile = tiles - 1; tile >= 0; --tile, t0 -= kTile, buf ^= 1) {
    float at[T][VEC], s[T][VEC], r[T][VEC], gsum[VEC], fwd[VEC], bwd[VEC], h[VEC];
    Raw<Act, VEC> xr[T], dor[T];
#pragma unroll
    for (int v = 0; v < VEC; ++v) gsum[v] = fwd[v] = bwd[v] = 0.0f, h[v] = next_h[v];
#pragma unroll
    for (int j = 0; j < T; ++j) {
      float gv[VEC], xv[VEC];
      xr[j] = next_x[j];
      dor[j] = next_o[j];
      next_g[j].get(gv);
      xr[j].get(xv);
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const Gate q = gate_of<SCALE>(gv[v]);
        at[j][v] = q.a;
        s[j][v] = q.s;
        r[j][v] = q.r;
        gsum[v] += gv[v];
        fwd[v] = fmaf(q.a, fwd[v], q.s * xv[v]);
      }
    }
#pragma unroll
    for (int j = T - 1; j >= 0; --j) {
      float dv[VEC];
      dor[j].get(dv);
#pragma unroll
      for (int v = 0; v < VEC; ++v) bwd[v] = at[j][v] * (dv[v] + bwd[v]);
    }
    load(t0 - kTile);
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      agg[buf][w][v][lane] = run_decay(gsum[v]);
      agg[buf][w][VEC + v][lane] = fwd[v];
      agg[buf][w][2 * VEC + v][lane] = bwd[v];
    }
    __syncthreads();
    float dc[VEC];  // the gradient that reaches the warp's last state from behind
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (i < w) h[v] = fmaf(agg[buf][i][v][lane], h[v], agg[buf][i][VEC + v][lane]);
    }
    if constexpr (CL > 1) {
      float pa[VEC], pb[VEC], ca[VEC], cb[VEC];
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        ca[v] = 1.0f;
        cb[v] = 0.0f;
#pragma unroll
        for (int i = W - 1; i >= 0; --i) {
          if (i == w) pa[v] = ca[v], pb[v] = cb[v];
          const float ai = agg[buf][i][v][lane];
          ca[v] *= ai;
          cb[v] = fmaf(ai, cb[v], agg[buf][i][2 * VEC + v][lane]);
        }
        if (w < CL) {
          cluster_store(&across[buf][rank][v][lane], w, ca[v]);
          cluster_store(&across[buf][rank][VEC + v][lane], w, cb[v]);
        }
      }
      cluster_barrier();
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
#pragma unroll
        for (int i = CL - 1; i >= 0; --i) {
          if (i == rank) dc[v] = fmaf(pa[v], carry[v], pb[v]);
          carry[v] = fmaf(across[buf][i][v][lane], carry[v], across[buf][i][VEC + v][lane]);
        }
      }
    } else {
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
#pragma unroll
        for (int i = W - 1; i >= 0; --i) {
          if (i == w) dc[v] = carry[v];
          carry[v] = fmaf(agg[buf][i][v][lane], carry[v], agg[buf][i][2 * VEC + v][lane]);
        }
      }
    }
    float before[T][VEC];
#pragma unroll
    for (int j = 0; j < T; ++j) {
      float xv[VEC];
      xr[j].get(xv);
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        before[j][v] = h[v];
        h[v] = fmaf(at[j][v], h[v], s[j][v] * xv[v]);
      }
    }
    auto wx = gx.row(t0 + T - 1);
    auto wg = gg.row(t0 + T - 1);
#pragma unroll
    for (int j = T - 1; j >= 0; --j, wx.prev(), wg.prev()) {
      float xv[VEC], dv[VEC], dx[VEC], dg[VEC];
      xr[j].get(xv);
      dor[j].get(dv);
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const float dh = dv[v] + dc[v];
        dx[v] = s[j][v] * dh;
        dc[v] = at[j][v] * dh;
        // a h dh + s' x dh, with s' = -a for 1 - a and -a^2 / s for sqrt(1 - a^2)
        float k = before[j][v];
        if constexpr (SCALE == GDN_SCALE_COMPLEMENT) k -= xv[v];
        if constexpr (SCALE == GDN_SCALE_SQRT) k = fmaf(-at[j][v] * r[j][v], xv[v], k);
        dg[v] = dc[v] * k;
      }
      if (live && t0 + j < len) {
        wx.store(dx);
        wg.store(dg);
      }
    }
  }
  if (a.hT && live && rank == 0 && w == 0) {
#pragma unroll
    for (int v = 0; v < VEC; ++v) a.hT[state + v] = carry[v];
  }
}

}  // namespace gdnq
