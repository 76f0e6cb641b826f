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

// v / scale as 8 e4m3 values. By the reciprocal, itself rounded once: a value within 2^-23 of itself of the border between
// two e4m3 values may go to either.
__device__ __forceinline__ uint2 pack_e4m3(const float (&v)[8], float scale) {
  const float r = 1.f / scale;
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i] * r, v[2 * i + 1] * r), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

}  // namespace mlora
