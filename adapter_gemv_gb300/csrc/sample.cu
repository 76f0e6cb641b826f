// sample.cu -- the next token of each row from a given random number, with temperature, top-k, top-p and min-p (sm_103a).
//
// First form: a CTA a row; each limit is a place in the row's order (logits descending, then ids), found by bisection of
// the order's code with a pass over the row for each of its bits.
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include <algorithm>

#include "sample_weight.cuh"

namespace mlora {

namespace {

constexpr int kThreads = 512;
constexpr int kIdBits = 19;
static_assert(MLORA_SAMPLE_MAX_VOCAB <= 1 << kIdBits, "ids fit the order's code");

template <int DT>
__device__ __forceinline__ float logit_at(const mlora_sampling &p, int64_t row, int t) {
  float x;
  if constexpr (DT == MLORA_FP32) x = static_cast<const float *>(p.logits)[row * p.ld + t];
  else x = Elem<DT>::lo(static_cast<const uint16_t *>(p.logits)[row * p.ld + t]);
  return x == x ? x + 0.f : -CUDART_INF_F;  // (-0 as 0)
}

// Place in the order: the larger logit first, then the lower id.
__device__ __forceinline__ uint64_t code_of(float x, int t) {
  const uint32_t b = __float_as_uint(x), up = b & 0x80000000u ? ~b : b | 0x80000000u;
  return (uint64_t)~up << kIdBits | (uint32_t)t;
}

__device__ __forceinline__ uint64_t sum_all(uint64_t v, uint64_t *part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
  __syncthreads();
  if (lane == 0) part[warp] = v;
  __syncthreads();
  v = lane < kThreads / 32 ? part[lane] : 0;
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
  return v;
}

template <int DT>
__global__ void __launch_bounds__(kThreads) sample_kernel(const __grid_constant__ mlora_sampling p, int32_t *status) {
  __shared__ float2 steps[kExp2Steps];
  __shared__ uint64_t part[32];
  __shared__ float tops[32];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const int r = p.row_request ? p.row_request[row] : (int)row;
  if (r == -1) return;
  if (r < -1 || r >= p.num_requests) {
    if (tid == 0) report(status, MLORA_STATUS_BAD_REQUEST);
    return;
  }
  for (int i = tid; i < kExp2Steps; i += kThreads) steps[i] = exp2_steps[i];
  float top = -CUDART_INF_F;
  for (int t = tid; t < p.vocab; t += kThreads) top = fmaxf(top, logit_at<DT>(p, row, t));
#pragma unroll
  for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
  if ((tid & 31) == 0) tops[tid >> 5] = top;
  __syncthreads();
  for (int i = 0; i < kThreads / 32; ++i) top = fmaxf(top, tops[i]);
  if (top == -CUDART_INF_F) {
    if (tid == 0) {
      p.token[row] = -1;
      if (p.logprob) p.logprob[row] = -CUDART_INF_F;
    }
    return;
  }
  const float temp = p.temperature ? p.temperature[r] : 1.f;
  const bool greedy = !(temp > 0.f);
  const WeightScale scale = weight_scale(greedy ? 1.f : temp);
  int k = p.top_k ? p.top_k[r] : 0;
  if (greedy) k = 1;
  if (k <= 0 || k > p.vocab) k = p.vocab;

  auto sum = [&](uint64_t last, bool mass) {  // over the order up to the code `last`
    uint64_t s = 0;
    for (int t = tid; t < p.vocab; t += kThreads) {
      const float x = logit_at<DT>(p, row, t);
      if (code_of(x, t) <= last) s += mass ? weight_of(x, top, scale, steps) : 1;
    }
    return sum_all(s, part);
  };
  auto place = [&](uint64_t least, bool mass) {  // the first code at which the sum reaches `least`
    uint64_t code = 0;
    for (int b = 31 + kIdBits; b >= 0; --b)
      if (sum(code | ((1ull << b) - 1), mass) < least) code |= 1ull << b;
    return code;
  };
  uint64_t kept = sum(k < p.vocab ? place(k, false) : ~0ull, true);
  const float tp = p.top_p ? p.top_p[r] : 1.f;
  if (tp < 1.f) kept = sum(place(max(times_ceil(fmaxf(tp, 0.f), kept), (uint64_t)1), true), true);
  const float mp = p.min_p ? p.min_p[r] : 0.f;
  if (mp > 0.f) {
    const float least = __double2float_ru((double)top + (double)temp * log((double)mp));
    uint64_t s = 0;
    for (int t = tid; t < p.vocab; t += kThreads) {
      const float x = logit_at<DT>(p, row, t);
      if (x >= least) s += weight_of(x, top, scale, steps);
    }
    kept = min(kept, max(sum_all(s, part), kWeightOne));
  }
  const float u = p.uniform[row];
  const uint64_t code = place(times_floor(u > 0.f ? fminf(u, 1.f - 0x1p-24f) : 0.f, kept) + 1, true);
  if (tid == 0) {
    const int t = (int)(code & ((1u << kIdBits) - 1));
    p.token[row] = t;
    if (p.logprob) {
      const float x = logit_at<DT>(p, row, t);
      float y = 0.f, yl = 0.f;
      if (x != top) weight_log2(x, top, scale, y, yl);
      const float more = (float)(kept - kWeightOne) * (1.f / (float)kWeightOne);
      p.logprob[row] = (y + yl) * 0.693147182f - log1pf(more);
    }
  }
}

template <int DT>
cudaError_t launch(const mlora_sampling &p, int32_t *status, cudaStream_t stream) {
  const cudaError_t e = launch_waiting(sample_kernel<DT>, dim3(p.num_rows), dim3(kThreads), 0, 1, stream, p, status);
  if (e == cudaSuccess) api_count_launch();
  return e;
}

}  // namespace

cudaError_t launch_sample(const mlora_sampling &p, int32_t *status, cudaStream_t stream) {
  switch (p.dtype) {
    case MLORA_FP32: return launch<MLORA_FP32>(p, status, stream);
    case MLORA_BF16: return launch<MLORA_BF16>(p, status, stream);
    default: return launch<MLORA_FP16>(p, status, stream);
  }
}

}  // namespace mlora
