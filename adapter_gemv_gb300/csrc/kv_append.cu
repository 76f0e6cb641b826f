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

#include <algorithm>

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

// A thread takes the same unit of ROWS rows, all loads on their way before the first store.
template <int DT, int ROWS>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const __grid_constant__ AppendParams p, int32_t *status) {
  pdl_wait();
  pdl_launch_dependents();
  const mlora_kv_rows &r = p.r;
  const int D = p.c.head_dim, hq = r.num_q_heads, hk = p.c.num_kv_heads, half = r.rotary_dim >> 1;
  const int u = blockIdx.x * kThreads + threadIdx.x;
  if (u >= p.per_row.d) return;
  // the unit: which of q, k, v, its head, and the head's elements it covers (the first of them)
  const int rot_units = (hq + hk) * p.per_head.d;
  const bool is_v = u >= rot_units;
  const FastDiv &per = is_v ? p.chunks : p.per_head;
  const int w0 = is_v ? u - rot_units : u;
  int h = div_by(per, w0);
  const int w = w0 - h * per.d;
  const bool is_q = !is_v && h < hq;
  if (!is_v && !is_q) h -= hq;
  const bool pairs = !is_v && w < p.pair_units;
  const int e = (pairs || is_v ? w : w + p.pair_units) * 8;  // a pair unit holds two chunks
  const bool turned = pairs || (!is_v && r.rope_interleaved && e < r.rotary_dim);
  const uint16_t *src = static_cast<const uint16_t *>(is_v ? r.v : is_q ? r.q : r.k) + (int64_t)h * D + e;
  const int64_t ld = is_v ? r.ldv : is_q ? r.ldq : r.ldk;

  int64_t slot[ROWS];
  int pos[ROWS];
  const int row0 = blockIdx.y * ROWS;
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int row = row0 + i;
    slot[i] = row < r.num_rows ? r.cache_slot[row] : -1;
    pos[i] = row < r.num_rows && r.rotary_dim ? r.position[row] : 0;
  }
  uint4 x[ROWS], y[ROWS];
  // Rows without a slot are loaded, too (the arrays have them): their slot is on its way. Waiting for it before the
  // loads: 164 us instead of 132 for 12604 rows, 29 instead of 24 for 2000; a row a thread, eight one after another
  // with the next slot fetched ahead: 136 and 28.
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    if (row0 + i >= r.num_rows) continue;
    x[i] = ldg_u4(src + (row0 + i) * ld);
    if (pairs) y[i] = ldg_u4(src + (row0 + i) * ld + half);
  }
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    int bad = 0;
    if (slot[i] < -1 || slot[i] >= p.slots) bad |= MLORA_STATUS_BAD_SLOT;
    if (slot[i] != -1 && r.rotary_dim && (pos[i] < 0 || pos[i] >= r.max_position)) bad |= MLORA_STATUS_BAD_LENGTH;
    if (bad && u == 0) report(status, bad);
    if (bad || slot[i] < 0) continue;
    if (turned) {
      const float *cs = r.rope_cos + (int64_t)pos[i] * half, *sn = r.rope_sin + (int64_t)pos[i] * half;
      float a[8], b[8];
      unpack8<DT>(x[i], a);
      if (pairs) {
        unpack8<DT>(y[i], b);
        rotate(a, b, cs + e, sn + e);
        y[i] = pack8<DT>(b);
      } else {
        const float4 c = *reinterpret_cast<const float4 *>(cs + e / 2), s = *reinterpret_cast<const float4 *>(sn + e / 2);
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x0 = a[2 * j], x1 = a[2 * j + 1];
          a[2 * j] = x0 * cc[j] - x1 * ss[j];
          a[2 * j + 1] = x1 * cc[j] + x0 * ss[j];
        }
      }
      x[i] = pack8<DT>(a);
    }
    uint16_t *dst;
    if (is_q) {
      dst = static_cast<uint16_t *>(r.q_out) + (row0 + i) * r.ldq_out + (int64_t)h * D + e;
    } else {
      const int64_t pg = p.slots <= INT32_MAX ? div_by(p.page, (int32_t)slot[i]) : slot[i] / p.page.d;
      dst = (is_v ? p.v : p.k) + pg * p.c.page_stride + (slot[i] - pg * p.page.d) * p.c.token_stride +
            h * p.c.head_stride + e;
    }
    *reinterpret_cast<uint4 *>(dst) = x[i];
    if (pairs) *reinterpret_cast<uint4 *>(dst + half) = y[i];
  }
}

template <int ROWS>
cudaError_t launch(const AppendParams &p, int32_t *status, cudaStream_t stream) {
  const dim3 grid((p.per_row.d + kThreads - 1) / kThreads, (p.r.num_rows + ROWS - 1) / ROWS);
  const cudaError_t e =
      p.c.dtype == MLORA_BF16
          ? launch_waiting(kv_append_kernel<MLORA_BF16, ROWS>, grid, dim3(kThreads), 0, 1, stream, p, status)
          : launch_waiting(kv_append_kernel<MLORA_FP16, ROWS>, grid, dim3(kThreads), 0, 1, stream, p, status);
  if (e == cudaSuccess) api_count_launch();
  return e;
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
  for (int64_t row0 = 0; row0 < r.num_rows; row0 += 65535) {  // (the last step may pass 2^31)
    AppendParams q = p;
    q.r.num_rows = (int32_t)std::min<int64_t>(65535, r.num_rows - row0);
    q.r.cache_slot += row0;
    if (q.r.position) q.r.position += row0;
    q.r.k = static_cast<const uint16_t *>(r.k) + row0 * r.ldk;
    q.r.v = static_cast<const uint16_t *>(r.v) + row0 * r.ldv;
    if (r.num_q_heads) {
      q.r.q = static_cast<const uint16_t *>(r.q) + row0 * r.ldq;
      q.r.q_out = static_cast<uint16_t *>(r.q_out) + row0 * r.ldq_out;
    }
    // Two rows a thread where that still leaves every SM its eight CTAs: 12604 rows of 40 + 80 heads of 128 take
    // 131 us so, 160 with a row each, 138 with four (5.9 TB/s of reads and writes; a copy reaches 6.7). 32
    // rows: 2.3 us with a row each.
    const cudaError_t e = (int64_t)q.r.num_rows * p.per_row.d >= (int64_t)sm_count() * 8 * kThreads * 2
                              ? launch<2>(q, status, stream) : launch<1>(q, status, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace mlora
