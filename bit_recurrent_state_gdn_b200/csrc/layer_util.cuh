// Device helpers shared by the operators around the recurrence.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "device_util.cuh"
#include "layer_args.h"

namespace gdnq {

// Tokens of sequence b.
__device__ __forceinline__ int seq_len(const int32_t* lens, int b, int L) {
  return lens ? min(max(lens[b], 0), L) : L;
}

// Offset of flat channel c = h D + d of sequence b's first token.
__device__ __forceinline__ int64_t channel_offset(const Tok& t, int b, int h, int d) {
  return (int64_t)b * t.sb + (int64_t)h * t.sh + d;
}

// Copies BYTES (4, 8 or 16) aligned bytes to shared memory asynchronously, or zeros where `ok` does
// not hold; `from` may be any valid address then, nothing is read.
template <int BYTES>
__device__ __forceinline__ void async_piece(uint32_t to, const void* from, bool ok) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(to), "l"(from),
                 "r"(ok ? 16 : 0)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;\n" ::"r"(to), "l"(from),
                 "r"(ok ? BYTES : 0), "n"(BYTES)
                 : "memory");
}

template <int BYTES>
__device__ __forceinline__ void async_piece(uint32_t to, const void* from) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(to), "l"(from) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"(to), "l"(from), "n"(BYTES)
                 : "memory");
}

// A kernel whose partial sums a second one adds lets that one be launched while it still runs; the
// second waits for all of the first one's work before it reads.
__device__ __forceinline__ void let_next_launch() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }
__device__ __forceinline__ void wait_for_last() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }

// 1 / sqrt(x) on the hardware path.
__device__ __forceinline__ float rsqrt_hw(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float sigmoidf(float u) { return __fdividef(1.0f, 1.0f + fast_exp(-u)); }

__device__ __forceinline__ F2 f2_all(float x) { return f2(x, x); }

__device__ __forceinline__ float rcp_hw(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// act(u), and act'(u) where it is asked for.
template <int ACT, bool SLOPE>
__device__ __forceinline__ void act_pair(F2 u, F2& v, F2& slope) {
  if constexpr (ACT == GDN_ACT_NONE) {
    v = u;
    slope = f2_all(1.0f);
  } else {
    float y0, y1, d0, d1;
    f2_get(f2_mul(u, f2_all(-1.4426950408889634f)), y0, y1);
    f2_get(f2_add(f2(exp2_hw(y0), exp2_hw(y1)), f2_all(1.0f)), d0, d1);
    const F2 q = f2(rcp_hw(d0), rcp_hw(d1));  // the sigmoid
    v = ACT == GDN_ACT_SILU ? f2_mul(u, q) : q;
    if constexpr (SLOPE) {
      const F2 rest = f2_fma(q, f2_all(-1.0f), f2_all(1.0f));
      slope = ACT == GDN_ACT_SILU ? f2_fma(v, rest, q) : f2_mul(q, rest);
    }
  }
}

}  // namespace gdnq
