// fp8_matmul.cu -- y = x W^T of e4m3 operands with a scale for each block of 128 (sm_103a).
//
// First form: a CTA a tile of 64 x 64, operands as fp32 in shared memory, fp32 products.
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "serve.cuh"

namespace mlora {

namespace {

constexpr int kTile = 64, kStep = 16, kThreads = 256;

__device__ __forceinline__ float e4m3_value(uint8_t b) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(b, __NV_E4M3)));
}

template <int DT>
__global__ void __launch_bounds__(kThreads) matmul_kernel(const __grid_constant__ mlora_matmul p) {
  __shared__ float xs[kStep][kTile + 1], ws[kStep][kTile + 1];
  pdl_wait();
  pdl_launch_dependents();
  const int n0 = blockIdx.x * kTile;
  const int64_t m0 = (int64_t)blockIdx.y * kTile;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16, lr = threadIdx.x / 4, lk = threadIdx.x % 4 * 4;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < p.d_in; k0 += MLORA_FP8_BLOCK) {
    float part[4][4] = {};
    const int k1 = min(k0 + MLORA_FP8_BLOCK, p.d_in);
    for (int k = k0; k < k1; k += kStep) {
      uint32_t xv = 0, wv = 0;
      if (m0 + lr < p.num_rows) xv = *reinterpret_cast<const uint32_t *>(static_cast<const uint8_t *>(p.x) + (m0 + lr) * p.ldx + k + lk);
      if (n0 + lr < p.d_out) wv = *reinterpret_cast<const uint32_t *>(static_cast<const uint8_t *>(p.w) + (int64_t)(n0 + lr) * p.ldw + k + lk);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        xs[lk + i][lr] = e4m3_value((uint8_t)(xv >> (8 * i)));
        ws[lk + i][lr] = e4m3_value((uint8_t)(wv >> (8 * i)));
      }
      __syncthreads();
#pragma unroll
      for (int kk = 0; kk < kStep; ++kk)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) part[i][j] = fmaf(xs[kk][ty * 4 + i], ws[kk][tx * 4 + j], part[i][j]);
    }
    const int b = k0 / MLORA_FP8_BLOCK;
    const float sw = p.w_scale[(int64_t)(n0 / MLORA_FP8_BLOCK) * p.ldws + b];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t m = m0 + ty * 4 + i;
      const float s = m < p.num_rows ? p.x_scale[m * p.ldxs + b] * sw : 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(s, part[i][j], acc[i][j]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t m = m0 + ty * 4 + i;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + tx * 4 + j;
      if (m < p.num_rows && n < p.d_out) static_cast<uint16_t *>(p.y)[m * p.ldy + n] = Elem<DT>::from_float(acc[i][j]);
    }
  }
}

}  // namespace

cudaError_t launch_fp8_matmul(const mlora_matmul &p, int32_t *status, cudaStream_t stream) {
  const int64_t most = 65535 * (int64_t)kTile;
  for (int64_t row0 = 0; row0 < p.num_rows; row0 += most) {
    mlora_matmul q = p;
    q.num_rows = (int32_t)std::min<int64_t>(most, p.num_rows - row0);
    q.x = static_cast<const uint8_t *>(p.x) + row0 * p.ldx;
    q.x_scale = p.x_scale + row0 * p.ldxs;
    q.y = static_cast<uint16_t *>(p.y) + row0 * p.ldy;
    const dim3 grid((q.d_out + kTile - 1) / kTile, (q.num_rows + kTile - 1) / kTile);
    const cudaError_t e = p.dtype == MLORA_BF16
                              ? launch_waiting(matmul_kernel<MLORA_BF16>, grid, dim3(kThreads), 0, 1, stream, q)
                              : launch_waiting(matmul_kernel<MLORA_FP16>, grid, dim3(kThreads), 0, 1, stream, q);
    if (e != cudaSuccess) return e;
    api_count_launch();
  }
  return cudaSuccess;
}

}  // namespace mlora
