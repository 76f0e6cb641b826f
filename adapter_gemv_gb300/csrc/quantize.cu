// quantize.cu -- 16-bit rows, or silu(gate) x of an MLP, as 8-bit rows (sm_103a).
//
// Elementwise but for the maximum of each block of 128, which half a warp holds: every element read once and
// written once; by launch and one load for a decode step's rows. Without a gate, 12604 x 4096 bf16 (157 MB): 40 us, bound by each thread's one
// trip to memory (of 15 cycles a warp and instruction 7 wait for it, at six CTAs an SM by 34 registers). silu(gate) x of 12604 x 13824
// with 16 and 8 bits out: 278 to 282 us, 4.4 TB/s, the schedulers 74 % busy with the exponential and the quotient, and the same trip. With
// __expf and __fdividef it takes 209 us, with expf and __fdividef 231: of 174 M values the 8-bit ones are as good (328 and 326 at the wrong neighbour, 334 with
// fp32's own exponential and quotient), but 470 and 461 of the 16-bit ones are rounded the wrong way, against 77 so and 123 of a plain fp32 form.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "rows8.cuh"

namespace mlora {

namespace {

constexpr int kThreads = 256;

// g / (1 + exp(-g)), by the exponential that is at most 1: of a far negative g it is what fp32 still holds.
__device__ __forceinline__ float silu(float g) {
  const float t = expf(-fabsf(g));
  return (g < 0.f ? g * t : g) / (1.f + t);
}

// Half warp u takes block u % blocks of row u / blocks.
template <int DT>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const __grid_constant__ mlora_quant p,
                                                            const __grid_constant__ FastDiv blocks) {
  pdl_wait();
  pdl_launch_dependents();
  const int u = (blockIdx.x * kThreads + threadIdx.x) / kBlockChunks;
  const int row = div_by(blocks, u), b = u - row * blocks.d;
  const int e = b * MLORA_FP8_BLOCK + threadIdx.x % kBlockChunks * 8;
  const bool in = row < p.num_rows && e < p.width;
  float v[8] = {};
  if (in) {
    unpack8<DT>(ldg_u4(static_cast<const uint16_t *>(p.x) + row * p.ldx + e), v);
    if (p.gate) {
      float g[8];
      unpack8<DT>(ldg_u4(static_cast<const uint16_t *>(p.gate) + row * p.ldg + e), g);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= silu(g[i]);
    }
    if (p.out) *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + row * p.ldo + e) = pack8<DT>(v);
  }
  if (p.q) {
    const float s = block_scale(v);
    if (in) {
      *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.q) + row * p.ldq + e) = pack_e4m3(v, s);
      if (threadIdx.x % kBlockChunks == 0) p.q_scale[row * p.lds + b] = s;
    }
  }
}

}  // namespace

cudaError_t launch_quantize(const mlora_quant &p, cudaStream_t stream) {
  const FastDiv blocks = fast_div((p.width + MLORA_FP8_BLOCK - 1) / MLORA_FP8_BLOCK);
  const int64_t most = std::max<int64_t>(1, (INT32_MAX - kThreads) / kBlockChunks / blocks.d);  // threads are counted in 31 bits
  for (int64_t row0 = 0; row0 < p.num_rows; row0 += most) {
    mlora_quant q = p;
    q.num_rows = (int32_t)std::min<int64_t>(most, p.num_rows - row0);
    q.x = static_cast<const uint16_t *>(p.x) + row0 * p.ldx;
    if (p.gate) q.gate = static_cast<const uint16_t *>(p.gate) + row0 * p.ldg;
    if (p.out) q.out = static_cast<uint16_t *>(p.out) + row0 * p.ldo;
    if (p.q) q.q = static_cast<uint8_t *>(p.q) + row0 * p.ldq, q.q_scale = p.q_scale + row0 * p.lds;
    const int64_t threads = (int64_t)q.num_rows * blocks.d * kBlockChunks;
    const dim3 grid((unsigned)((threads + kThreads - 1) / kThreads));
    const cudaError_t e = p.dtype == MLORA_BF16
                              ? launch_waiting(quantize_kernel<MLORA_BF16>, grid, dim3(kThreads), 0, 1, stream, q, blocks)
                              : launch_waiting(quantize_kernel<MLORA_FP16>, grid, dim3(kThreads), 0, 1, stream, q, blocks);
    if (e != cudaSuccess) return e;
    api_count_launch();
  }
  return cudaSuccess;
}

}  // namespace mlora
