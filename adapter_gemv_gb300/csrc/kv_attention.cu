// kv_attention.cu -- attention of new tokens over the paged key-value cache (sm_103a).
//
//   s_t = scale q.K_t,  m = max_t s_t,  l = sum_t exp(s_t - m),  out = sum_t exp(s_t - m) V_t / l
// in one pass over the tokens: a running maximum m, and l and out rescaled by exp(m - m') when it grows.
// Parts of the tokens are joined with the same rescaling.
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "serve.cuh"

namespace mlora {

namespace {

constexpr int kThreads = 128;

struct AttnParams {
  mlora_kv_cache c;
  mlora_kv_attn a;
  const uint16_t *k, *v;
  FastDiv page;
};

// A CTA per (row, query head), a warp per token, a lane per 16-byte chunk of the head.
template <int DT>
__global__ void __launch_bounds__(kThreads) kv_attention_kernel(const __grid_constant__ AttnParams p, int32_t row0,
                                                                int32_t *status) {
  __shared__ float sm[4], sl[4], so[4][MLORA_KV_MAX_HEAD_DIM];
  pdl_wait();
  const mlora_kv_attn &a = p.a;
  const int D = p.c.head_dim, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = (int64_t)row0 + blockIdx.y;
  const int h = blockIdx.x, hk = h / (a.num_q_heads / p.c.num_kv_heads);
  const int req = a.row_request ? a.row_request[row] : (int)row;
  const int pos = a.position[row];
  int bad = 0;
  if (pos < -1 || pos >= (int64_t)a.max_pages * p.page.d) bad |= MLORA_STATUS_BAD_LENGTH;
  if (pos >= 0 && (req < 0 || req >= a.num_requests)) bad |= MLORA_STATUS_BAD_REQUEST;
  if (bad) {
    if (threadIdx.x == 0) report(status, bad);
    return;
  }
  const int first = a.window ? max(0, pos + 1 - a.window) : 0;
  const bool on = lane * 8 < D;
  float q[8] = {}, o[8] = {}, m = -CUDART_INF_F, l = 0.f;
  if (on) unpack8<DT>(ldg_u4(static_cast<const uint16_t *>(a.q) + row * a.ldq + (int64_t)h * D + lane * 8), q);
  for (int t = first + warp; t <= pos; t += 4) {
    const int pg = div_by(p.page, t);
    const int id = a.page_table[(int64_t)req * a.table_stride + pg];
    if (id < 0 || id >= p.c.num_pages) {
      if (lane == 0) report(status, MLORA_STATUS_BAD_PAGE);
      continue;
    }
    const int64_t at = (int64_t)id * p.c.page_stride + (int64_t)(t - pg * p.page.d) * p.c.token_stride +
                       hk * p.c.head_stride + lane * 8;
    float k[8] = {}, v[8] = {};
    if (on) {
      unpack8<DT>(ldg_u4(p.k + at), k);
      unpack8<DT>(ldg_u4(p.v + at), v);
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += q[i] * k[i];
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
    s *= a.scale;
    const float m2 = fmaxf(m, s), keep = m2 == -CUDART_INF_F ? 1.f : expf(m - m2);
    const float w = m2 == -CUDART_INF_F ? 0.f : expf(s - m2);
    l = l * keep + w;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = o[i] * keep + w * v[i];
    m = m2;
  }
  if (lane == 0) sm[warp] = m, sl[warp] = l;
  if (on)
#pragma unroll
    for (int i = 0; i < 8; ++i) so[warp][lane * 8 + i] = o[i];
  __syncthreads();
  const float top = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  const float base = top == -CUDART_INF_F ? 0.f : top;
  float sum = 0.f;
  for (int w = 0; w < 4; ++w) sum += sl[w] * expf(sm[w] - base);
  for (int d = threadIdx.x; d < D; d += kThreads) {
    float f = 0.f;
    for (int w = 0; w < 4; ++w) f += so[w][d] * expf(sm[w] - base);
    static_cast<uint16_t *>(a.out)[row * a.ldo + (int64_t)h * D + d] = Elem<DT>::from_float(sum == 0.f ? 0.f : f / sum);
  }
  if (a.lse && threadIdx.x == 0) a.lse[row * a.num_q_heads + h] = sum == 0.f ? -CUDART_INF_F : base + logf(sum);
}

}  // namespace

int64_t kv_attention_workspace_bytes(int32_t) { return 16; }

cudaError_t launch_kv_attention(const mlora_kv_cache &c, const mlora_kv_attn &a, int32_t layer, int32_t *status,
                                cudaStream_t stream) {
  AttnParams p{};
  p.c = c;
  p.a = a;
  p.k = static_cast<const uint16_t *>(c.k) + layer * c.layer_stride;
  p.v = static_cast<const uint16_t *>(c.v) + layer * c.layer_stride;
  p.page = fast_div(c.page_tokens);
  for (int32_t row0 = 0; row0 < a.num_rows; row0 += 65535) {
    const dim3 grid(a.num_q_heads, min(65535, a.num_rows - row0));
    const cudaError_t e =
        c.dtype == MLORA_BF16
            ? launch_waiting(kv_attention_kernel<MLORA_BF16>, grid, dim3(kThreads), 0, 1, stream, p, row0, status)
            : launch_waiting(kv_attention_kernel<MLORA_FP16>, grid, dim3(kThreads), 0, 1, stream, p, row0, status);
    if (e != cudaSuccess) return e;
    api_count_launch();
  }
  return cudaSuccess;
}

}  // namespace mlora
