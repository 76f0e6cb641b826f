// logits_adjust.cu -- each request's penalties, biases, temperature and grammar mask on its logits (sm_103a).
//
// Elementwise over [rows][vocab] once the history is a count per token: 2 x 4 bytes a logit and a
// mask bit against a handful of flops, so bound by memory for a batch and by latency for a row.
//
// A CTA takes a slice of one row's vocabulary. It starts the loads of its logits into registers, then
// counts the history's tokens that fall in its slice in shared memory (whole-number atomics: the
// order does not matter), and applies the formula to what it holds. Each CTA of a row reads the
// whole history (at most some 16 KB, from L2 after the first), which is cheaper than a
// counting kernel before this one or an array of counts in global memory.
// A count word holds the occurrences past the prompt, and bit 31 for a token of the prompt. Of several
// bias entries with one id the last has to win: the bias word is the largest entry number + 1.
//
// Rows of an odd vocabulary start at any multiple of the element: a slice is cut where 16-byte
// vectors are aligned in memory, counted from the aligned address before the row's start.
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "serve.cuh"

namespace mlora {

namespace {

constexpr int kThreads = 256;
constexpr uint32_t kInPrompt = 0x80000000u;

template <int DT>
struct Vec {  // a 16-byte vector of logits
  static constexpr int N = 8;
  using T = uint16_t;
  static __device__ __forceinline__ void unpack(const uint4 &u, float (&f)[N]) { unpack8<DT>(u, f); }
  static __device__ __forceinline__ uint4 pack(const float (&f)[N]) { return pack8<DT>(f); }
  static __device__ __forceinline__ float get(T w) { return Elem<DT>::lo(w); }
  static __device__ __forceinline__ T put(float f) { return Elem<DT>::from_float(f); }
};
template <>
struct Vec<MLORA_FP32> {
  static constexpr int N = 4;
  using T = float;
  static __device__ __forceinline__ void unpack(const uint4 &u, float (&f)[N]) {
    f[0] = __uint_as_float(u.x), f[1] = __uint_as_float(u.y), f[2] = __uint_as_float(u.z), f[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[N]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
  static __device__ __forceinline__ float get(T w) { return w; }
  static __device__ __forceinline__ T put(float f) { return f; }
};

template <int DT, int NV>  // NV vectors a thread
__global__ void __launch_bounds__(kThreads) logits_kernel(const __grid_constant__ mlora_logits p, int32_t row0,
                                                          int32_t *status) {
  using V = Vec<DT>;
  using T = typename V::T;
  constexpr int kSlice = kThreads * NV * V::N;
  extern __shared__ __align__(16) uint32_t tab[];  // [kSlice] counts (with a history), [kSlice] biases (with a list)
  pdl_wait();
  const int tid = threadIdx.x, slice = blockIdx.x;
  const int64_t row = (int64_t)row0 + blockIdx.y;
  int bad = 0;
  const int r = p.row_request ? p.row_request[row] : (int)row;
  if (r < -1 || r >= p.num_requests) bad |= MLORA_STATUS_BAD_REQUEST;
  int total = 0, prompt = 0, bias0 = 0, bias1 = 0, grammar = -1;
  float rep = 1.f, pres = 0.f, freq = 0.f, temp = 0.f;
  if (!bad && r >= 0) {
    if (p.total_len) {
      total = p.total_len[r], prompt = p.prompt_len[r];
      if (total < 0 || total > p.tokens_stride || prompt < 0 || prompt > total) bad |= MLORA_STATUS_BAD_LENGTH;
    }
    if (p.bias_offsets) {
      bias0 = p.bias_offsets[r], bias1 = p.bias_offsets[r + 1];
      if (bias0 < 0 || bias1 < bias0 || bias1 > p.num_bias) bad |= MLORA_STATUS_BAD_LENGTH;
    }
    if (p.mask) {
      grammar = p.mask_index[r];
      if (grammar < -1 || grammar >= p.num_masks) bad |= MLORA_STATUS_BAD_SLOT;
    }
    if (p.repetition) rep = p.repetition[r];
    if (p.presence) pres = p.presence[r];
    if (p.frequency) freq = p.frequency[r];
    if (p.temperature) temp = p.temperature[r];
  }
  if (bad && slice == 0 && tid == 0) report(status, bad);
  if (bad || r < 0) return;

  const T *src = static_cast<const T *>(p.logits) + row * p.ld;
  T *dst = static_cast<T *>(p.out) + row * p.ldo;
  const int skew = (int)((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(T));  // elements before the row's start
  const bool same_skew = (int)((reinterpret_cast<uintptr_t>(dst) & 15) / sizeof(T)) == skew;
  const int first = slice * kSlice - skew;  // token of the slice's first place (below 0 in a skewed first slice)
  if (first >= p.vocab) return;

  float x[NV][V::N];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int t = first + (k * kThreads + tid) * V::N;
    if (t >= 0 && t + V::N <= p.vocab) {
      V::unpack(ldg_u4(src + t), x[k]);
    } else {
#pragma unroll
      for (int e = 0; e < V::N; ++e) x[k][e] = (t + e >= 0 && t + e < p.vocab) ? V::get(src[t + e]) : 0.f;
    }
  }

  const bool counted = total > 0, biased = bias1 > bias0;
  uint32_t *count = tab, *entry = tab + (p.total_len ? kSlice : 0);
  if (counted || biased) {
    for (int i = tid * 4; i < kSlice; i += kThreads * 4) {
      if (counted) *reinterpret_cast<uint4 *>(count + i) = make_uint4(0, 0, 0, 0);
      if (biased) *reinterpret_cast<uint4 *>(entry + i) = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    const int32_t *text = p.tokens + (int64_t)r * p.tokens_stride;
    int wrong = 0;
#pragma unroll 4
    for (int i = tid; i < total; i += kThreads) {
      const int t = text[i];
      if ((uint32_t)t >= (uint32_t)p.vocab) {
        wrong = MLORA_STATUS_BAD_TOKEN;
        continue;
      }
      const uint32_t at = (uint32_t)(t - first);
      if (at < (uint32_t)kSlice) {
        if (i < prompt) atomicOr(count + at, kInPrompt);
        else atomicAdd(count + at, 1u);
      }
    }
    for (int i = bias0 + tid; i < bias1; i += kThreads) {
      const int t = p.bias_token[i];
      if ((uint32_t)t >= (uint32_t)p.vocab) {
        wrong = MLORA_STATUS_BAD_TOKEN;
        continue;
      }
      const uint32_t at = (uint32_t)(t - first);
      if (at < (uint32_t)kSlice) atomicMax(entry + at, (uint32_t)(i - bias0) + 1u);
    }
    if (wrong && slice == 0) report(status, wrong);
    __syncthreads();
  }

  const uint32_t *bits = grammar >= 0 ? p.mask + grammar * p.mask_stride : nullptr;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int at = (k * kThreads + tid) * V::N, t = first + at;
#pragma unroll
    for (int e = 0; e < V::N; ++e) {
      float f = x[k][e];
      if (counted) {
        const uint32_t c = count[at + e];
        if (c) f = f > 0.f ? f / rep : f * rep;
        const uint32_t made = c & ~kInPrompt;
        if (made) f = f - freq * (float)made - pres;
      }
      if (biased) {
        const uint32_t b = entry[at + e];
        if (b) f += p.bias_value[bias0 + b - 1];
      }
      if (temp > 0.f) f = f / temp;
      if (bits && t + e >= 0 && t + e < p.vocab && !((bits[(t + e) >> 5] >> ((t + e) & 31)) & 1u)) f = -CUDART_INF_F;
      x[k][e] = f;
    }
    if (same_skew && t >= 0 && t + V::N <= p.vocab) {
      *reinterpret_cast<uint4 *>(dst + t) = V::pack(x[k]);
    } else {
#pragma unroll
      for (int e = 0; e < V::N; ++e)
        if (t + e >= 0 && t + e < p.vocab) dst[t + e] = V::put(x[k][e]);
    }
  }
}

template <int DT, int NV>
cudaError_t launch(const mlora_logits &a, int32_t *status, cudaStream_t stream) {
  constexpr int kSlice = kThreads * NV * Vec<DT>::N;
  const size_t smem = ((a.total_len ? 1 : 0) + (a.bias_offsets ? 1 : 0)) * kSlice * sizeof(uint32_t);
  cudaError_t e = cudaFuncSetAttribute(logits_kernel<DT, NV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       2 * kSlice * (int)sizeof(uint32_t));
  if (e != cudaSuccess) return e;
  // a row may start up to one vector's elements after an aligned address
  const int64_t slices = ((int64_t)a.vocab + Vec<DT>::N - 1 + kSlice - 1) / kSlice;
  for (int32_t row0 = 0; row0 < a.num_rows; row0 += 65535) {
    const dim3 grid((unsigned)slices, (unsigned)min(65535, a.num_rows - row0));
    e = launch_waiting(logits_kernel<DT, NV>, grid, dim3(kThreads), smem, 1, stream, a, row0, status);
    if (e != cudaSuccess) return e;
    api_count_launch();
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_logits_adjust(const mlora_logits &a, int32_t *status, cudaStream_t stream) {
  switch (a.dtype) {
    case MLORA_FP32: return launch<MLORA_FP32, 4>(a, status, stream);
    case MLORA_BF16: return launch<MLORA_BF16, 2>(a, status, stream);
    default: return launch<MLORA_FP16, 2>(a, status, stream);
  }
}

}  // namespace mlora
