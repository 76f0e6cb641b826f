// rms_norm.cu -- the residual's addition, the root-mean-square norm and its 8-bit rows in one pass (sm_103a).
//
// Per row: h = x + residual, v = weight h / sqrt(mean h^2 + eps). h stays in registers between the row's sum
// and its use, so that every element is read once and written once per output; a handful of flops a byte: bound by
// memory for a prompt's rows, by launch, one load and the row's sum for a decode step's.
//
// A CTA takes a row, a thread chunks of 8 elements, CTA width apart: the 16 lanes of half a warp hold a block of
// the 8-bit rows. 12604 rows of 5120 with a residual, 16 and 8 bits out (9 bytes an element): 112 us, 5.2 TB/s; 32 x 4096: 2.5 us.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "rows8.cuh"

namespace mlora {

namespace {

__device__ __forceinline__ float block_sum(float s, float *part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
  if (lane == 0) part[warp] = s;
  __syncthreads();
  s = lane < warps ? part[lane] : 0.f;
#pragma unroll
  for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
  return s;
}

template <int DT, int CH>  // CH chunks a thread
__global__ void __launch_bounds__(1024) rms_norm_kernel(const __grid_constant__ mlora_norm p) {
  __shared__ float part[2][32];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t row = blockIdx.x;
  const uint16_t *x = static_cast<const uint16_t *>(p.x) + row * p.ldx;
  const uint16_t *res = static_cast<const uint16_t *>(p.residual) + row * p.ldr;
  float h[CH][8];  // half of x + residual, which may pass fp32's range: halves of 16-bit numbers are exact, so is 2 h below it
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int e = (c * blockDim.x + threadIdx.x) * 8;
    if (e < p.width) {
      unpack8<DT>(ldg_u4(x + e), h[c]);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[c][i] *= 0.5f;
      if (p.residual) {
        float r[8];
        unpack8<DT>(ldg_u4(res + e), r);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[c][i] = fmaf(0.5f, r[i], h[c][i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) h[c][i] = 0.f;
    }
  }
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(h[c][i], h[c][i], s);
  s = block_sum(s, part[0]);
  float scale = 2.f, mean = 4.f * s / (float)p.width + p.eps;
  if (isinf(mean)) {  // squares, or eps, beyond fp32's range (or an infinity in the row): summed as those of h 2^-72
    scale = 0x1p-72f;
    s = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) s = fmaf(h[c][i] * scale, h[c][i] * scale, s);
    mean = block_sum(s, part[1]) / (float)p.width + p.eps * 0x1p-146f;  // (h is a half)
  }
  const float r = 1.f / sqrtf(mean);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int e = (c * blockDim.x + threadIdx.x) * 8;
    const bool in = e < p.width;
    float v[8];
    if (in && p.residual) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = h[c][i] + h[c][i];
      *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.residual_out) + row * p.ldro + e) = pack8<DT>(v);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = h[c][i] * scale * r;
    if (in && p.weight) {
      float w[8];
      unpack8<DT>(ldg_u4(static_cast<const uint16_t *>(p.weight) + e), w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= w[i];
    }
    if (in && p.out) *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + row * p.ldo + e) = pack8<DT>(v);
    if (p.q) {
      if (!in) {  // (columns behind the row have no part, whatever the row's sum)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
      }
      const float bs = block_scale(v);
      if (in) {
        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.q) + row * p.ldq + e) = pack_e4m3(v, bs);
        if (threadIdx.x % kBlockChunks == 0) p.q_scale[row * p.lds + e / MLORA_FP8_BLOCK] = bs;
      }
    }
  }
}

template <int DT, int CH>
cudaError_t launch(const mlora_norm &p, int threads, cudaStream_t stream) {
  const cudaError_t e = launch_waiting(rms_norm_kernel<DT, CH>, dim3(p.num_rows), dim3(threads), 0, 1, stream, p);
  if (e == cudaSuccess) api_count_launch();
  return e;
}

template <int DT>
cudaError_t dispatch(const mlora_norm &p, cudaStream_t stream) {
  const int chunks = p.width / 8;
  // One chunk a thread as far as a CTA goes: 12604 x 5120 take 112 us so, 121 with two, 133 with four; 32 x 4096 2.5, 3.5, 5.2
  const int ch = chunks <= 1024 ? 1 : chunks <= 2048 ? 2 : 4;
  const int threads = ((chunks + ch - 1) / ch + 31) & ~31;
  if (ch == 1) return launch<DT, 1>(p, threads, stream);
  if (ch == 2) return launch<DT, 2>(p, threads, stream);
  return launch<DT, 4>(p, threads, stream);
}

}  // namespace

cudaError_t launch_rms_norm(const mlora_norm &p, cudaStream_t stream) {
  return p.dtype == MLORA_BF16 ? dispatch<MLORA_BF16>(p, stream) : dispatch<MLORA_FP16>(p, stream);
}

}  // namespace mlora
