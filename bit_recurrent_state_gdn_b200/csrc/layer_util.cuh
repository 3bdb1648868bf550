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

// 1 / sqrt(x) on the hardware path.
__device__ __forceinline__ float rsqrt_hw(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float sigmoidf(float u) { return __fdividef(1.0f, 1.0f + fast_exp(-u)); }

}  // namespace gdnq
