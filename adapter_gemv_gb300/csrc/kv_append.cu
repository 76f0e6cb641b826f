// kv_append.cu -- rotary positions and the write of new k and v rows into the paged cache (sm_103a).
//
// Per row: q and k heads rotated in pairs, (a, b) -> (a c - b s, b c + a s) in fp32 with one rounding,
// v copied; k and v go to their cache slot. Every element is read once and written once, 2 flops a
// byte: bound by memory for a prompt's rows, by launch and two dependent loads (slot and position,
// then the tables) for a decode step's.
//
// A unit is what one thread does: the two 16-byte chunks that hold eight pairs (m, m + rot/2), or
// one 16-byte chunk of interleaved pairs, or one chunk that is copied. Units are numbered over rows,
// then heads, so neighbouring threads take neighbouring chunks.
#include <cuda_runtime.h>
#include <stdint.h>

#include "serve.cuh"

namespace mlora {

namespace {

constexpr int kThreads = 256;

struct AppendParams {
  mlora_kv_cache c;
  mlora_kv_rows r;
  uint16_t *k, *v;      // the layer's part of the cache
  FastDiv per_row;      // units of a row
  FastDiv per_head;     // units of a rotated head (q, k)
  FastDiv chunks;       // 16-byte chunks of a head
  FastDiv page;         // tokens of a page
  int32_t pair_units;   // units of a rotated head that hold half-split pairs
  int64_t slots;        // num_pages * page_tokens
};

template <int DT>
__device__ __forceinline__ void rotate(float (&a)[8], float (&b)[8], const float *cs, const float *sn) {
  float c[8], s[8];
  *reinterpret_cast<float4 *>(c) = reinterpret_cast<const float4 *>(cs)[0];
  *reinterpret_cast<float4 *>(c + 4) = reinterpret_cast<const float4 *>(cs)[1];
  *reinterpret_cast<float4 *>(s) = reinterpret_cast<const float4 *>(sn)[0];
  *reinterpret_cast<float4 *>(s + 4) = reinterpret_cast<const float4 *>(sn)[1];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = a[i], y = b[i];
    a[i] = x * c[i] - y * s[i];
    b[i] = y * c[i] + x * s[i];
  }
}

template <int DT>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const __grid_constant__ AppendParams p, int32_t *status) {
  pdl_wait();
  pdl_launch_dependents();
  const mlora_kv_rows &r = p.r;
  const int D = p.c.head_dim, hq = r.num_q_heads, hk = p.c.num_kv_heads;
  const int row = blockIdx.y;
  const int u = blockIdx.x * kThreads + threadIdx.x;
  if (u >= p.per_row.d) return;
  const int64_t slot = r.cache_slot[row];
  const int pos = r.rotary_dim ? r.position[row] : 0;
  int bad = 0;
  if (slot < -1 || slot >= p.slots) bad |= MLORA_STATUS_BAD_SLOT;
  if (slot != -1 && r.rotary_dim && (pos < 0 || pos >= r.max_position)) bad |= MLORA_STATUS_BAD_LENGTH;
  if (bad && u == 0) report(status, bad);
  if (bad || slot < 0) return;

  const int rot_units = (hq + hk) * p.per_head.d;
  const int64_t pg = slot / p.page.d;
  const int64_t cell = pg * p.c.page_stride + (slot - pg * p.page.d) * p.c.token_stride;
  if (u < rot_units) {
    int h = div_by(p.per_head, u);
    const int w = u - h * p.per_head.d;
    const uint16_t *src;
    uint16_t *dst;
    if (h < hq) {
      src = static_cast<const uint16_t *>(r.q) + row * r.ldq + (int64_t)h * D;
      dst = static_cast<uint16_t *>(r.q_out) + row * r.ldq_out + (int64_t)h * D;
    } else {
      h -= hq;
      src = static_cast<const uint16_t *>(r.k) + row * r.ldk + (int64_t)h * D;
      dst = p.k + cell + h * p.c.head_stride;
    }
    const int half = r.rotary_dim >> 1;
    if (w < p.pair_units) {
      const int e = w * 8;
      float a[8], b[8];
      unpack8<DT>(ldg_u4(src + e), a);
      unpack8<DT>(ldg_u4(src + e + half), b);
      rotate<DT>(a, b, r.rope_cos + (int64_t)pos * half + e, r.rope_sin + (int64_t)pos * half + e);
      *reinterpret_cast<uint4 *>(dst + e) = pack8<DT>(a);
      *reinterpret_cast<uint4 *>(dst + e + half) = pack8<DT>(b);
    } else {
      const int e = (w + p.pair_units) * 8;  // a pair unit holds two chunks
      uint4 x = ldg_u4(src + e);
      if (r.rope_interleaved && e < r.rotary_dim) {
        float f[8];
        unpack8<DT>(x, f);
        const float4 c = *reinterpret_cast<const float4 *>(r.rope_cos + (int64_t)pos * half + e / 2);
        const float4 s = *reinterpret_cast<const float4 *>(r.rope_sin + (int64_t)pos * half + e / 2);
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x0 = f[2 * i], x1 = f[2 * i + 1];
          f[2 * i] = x0 * cc[i] - x1 * ss[i];
          f[2 * i + 1] = x1 * cc[i] + x0 * ss[i];
        }
        x = pack8<DT>(f);
      }
      *reinterpret_cast<uint4 *>(dst + e) = x;
    }
  } else {
    const int w = u - rot_units;
    const int h = div_by(p.chunks, w), e = (w - h * p.chunks.d) * 8;
    *reinterpret_cast<uint4 *>(p.v + cell + h * p.c.head_stride + e) =
        ldg_u4(static_cast<const uint16_t *>(r.v) + row * r.ldv + (int64_t)h * D + e);
  }
}

}  // namespace

cudaError_t launch_kv_append(const mlora_kv_cache &c, const mlora_kv_rows &r, int32_t layer, int32_t *status,
                             cudaStream_t stream) {
  AppendParams p{};
  p.c = c;
  p.r = r;
  p.k = static_cast<uint16_t *>(c.k) + layer * c.layer_stride;
  p.v = static_cast<uint16_t *>(c.v) + layer * c.layer_stride;
  const int chunks = c.head_dim / 8;
  p.pair_units = r.rope_cos && !r.rope_interleaved ? r.rotary_dim / 16 : 0;
  p.per_head = fast_div(chunks - p.pair_units);
  p.chunks = fast_div(chunks);
  p.page = fast_div(c.page_tokens);
  p.slots = (int64_t)c.num_pages * c.page_tokens;
  p.per_row = fast_div((r.num_q_heads + c.num_kv_heads) * p.per_head.d + c.num_kv_heads * chunks);
  for (int32_t row0 = 0; row0 < r.num_rows; row0 += 65535) {
    AppendParams q = p;
    const int n = min(65535, r.num_rows - row0);
    q.r.cache_slot += row0;
    if (q.r.position) q.r.position += row0;
    q.r.k = static_cast<const uint16_t *>(r.k) + row0 * r.ldk;
    q.r.v = static_cast<const uint16_t *>(r.v) + row0 * r.ldv;
    if (r.num_q_heads) {
      q.r.q = static_cast<const uint16_t *>(r.q) + row0 * r.ldq;
      q.r.q_out = static_cast<uint16_t *>(r.q_out) + row0 * r.ldq_out;
    }
    const dim3 grid((p.per_row.d + kThreads - 1) / kThreads, n);
    const cudaError_t e = c.dtype == MLORA_BF16
                              ? launch_waiting(kv_append_kernel<MLORA_BF16>, grid, dim3(kThreads), 0, 1, stream, q, status)
                              : launch_waiting(kv_append_kernel<MLORA_FP16>, grid, dim3(kThreads), 0, 1, stream, q, status);
    if (e != cudaSuccess) return e;
    api_count_launch();
  }
  return cudaSuccess;
}

}  // namespace mlora
