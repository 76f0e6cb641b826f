// rows8.cuh -- 8-bit rows: e4m3 values with an fp32 scale for every block of 128 columns (sm_103a).
//
// A block's 16 chunks of 8 elements are held by the 16 lanes of half a warp.
#pragma once

#include <cuda_fp8.h>

#include "serve.cuh"

namespace mlora {

constexpr int kBlockChunks = MLORA_FP8_BLOCK / 8;
constexpr float kFp8Max = 448.f;
constexpr float kScaleMin = 1.17549435e-38f;  // 2^-126: its reciprocal is finite, and so is that of every scale above

// The larger of two, NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Scale of the block that the 16 lanes of a half warp hold 8 values each of (0 where there are none).
__device__ __forceinline__ float block_scale(const float (&v)[8]) {
  float m = fabsf(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max_nan(m, fabsf(v[i]));
#pragma unroll
  for (int d = kBlockChunks / 2; d; d >>= 1) m = max_nan(m, __shfl_xor_sync(~0u, m, d));
  return max_nan(m / kFp8Max, kScaleMin);
}

// v / scale as 8 e4m3 values: the fp32 quotient to the nearest, ties to even. A 16-bit v often is half way between two of
// them, so this is no product with a rounded 1 / scale: r + rest is 1 / scale to 2^-47 (the remainder 1 - r scale is exact by an fma), and v r +
// v rest, rounded once, is the quotient that a division rounds to: the same e4m3 for every pair of 16-bit significands
// of v and of the block's largest. 12604 x 4096 bf16: 40.1 us, 47.2 with eight divisions a thread, 38.3 with r alone, which takes 27 times
// as many values to the wrong neighbour as a division does (12 700 against 470 of 25.6 M).
__device__ __forceinline__ uint2 pack_e4m3(const float (&v)[8], float scale) {
  const float r = 1.f / scale;
  const float rest = r > 0.f ? fmaf(-r, scale, 1.f) * r : 0.f;  // (0: an infinite scale)
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = fmaf(v[i], r, v[i] * rest);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __nv_cvt_float2_to_fp8x2(make_float2(q[2 * i], q[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

}  // namespace mlora
