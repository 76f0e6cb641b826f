// kv_attention.cu -- attention of new tokens over the paged key-value cache (sm_103a).
//
//   s_t = scale q.K_t,  m = max_t s_t,  l = sum_t exp(s_t - m),  out = sum_t exp(s_t - m) V_t / l
// in one pass over the tokens: a running maximum m, and l and out rescaled by exp(m - m') when it grows.
// Parts of the tokens are joined with the same rescaling.
//
// Bound by memory: 4 bytes of K and V against 4 flops per query head of a group and token, so with at
// most 16 heads a group the matrix instructions are nearly idle and everything is about keeping
// loads in flight. Therefore:
//   * A warp works alone. It streams tiles of 16 tokens of one key-value head through a ring of its own
//     in shared memory (16-byte cp.async, three tiles of 8 KB at 128 elements a head: some 130 KB on
//     their way per SM), with no barrier between warps in the loop.
//   * The unit of work is a tile, not a request: the tiles of all rows and key-value heads form one
//     list, cut evenly over the SMs and over their warps, so the lengths do not have to match anything and one
//     long request fills the GPU as well as many short ones. A warp goes from one (row, head) to the
//     next without draining its ring.
//   * A (row, head) cut between warps is joined in two steps, in a fixed order: the warps of a CTA,
//     then the CTAs, by the one that finishes last (a counter that it returns to zero).
// The heads of a group are the rows of the matrix product (m16n8k16). With at most 8 the second half of
// the rows is free: the weights, which are rounded to 16 bits for the second product, are given there as the
// rounding's remainder, so that weight and remainder both meet V and nothing but fp32's error is left.
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "serve.cuh"
#include "tc.cuh"

namespace mlora {

namespace {

constexpr int kTile = 16;          // tokens of a tile
constexpr int kRowsPerLaunch = 1024;
constexpr int kMinTiles = 4;       // a warp's share of a small call, so that few pieces have to be joined
constexpr int kMaxGroup = 16;      // query heads of a work item

constexpr int attn_warps(int dp) { return dp == 256 ? 4 : 8; }
constexpr int attn_stages(int dp) { return dp == 64 ? 6 : 3; }
// Floats of a partial result: out [16][dp], then m [16] and l [16].
constexpr int partial_floats(int dp) { return kMaxGroup * (dp + 2); }
// Partial results of a CTA in the workspace: two a warp, two of its own.
constexpr int partial_slots(int dp) { return 2 * attn_warps(dp) + 2; }
constexpr int padded_dim(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

struct AttnParams {
  mlora_kv_cache c;
  mlora_kv_attn a;
  const uint16_t *k, *v;  // the layer's part of the cache
  FastDiv page;
  int32_t row0, rows;     // this launch's rows
  int32_t group, chunks;  // query heads of a key-value head, in chunks of at most 16
  float scale_log2;       // scale * log2(e)
  int32_t *counters;      // [CTAs], zero between calls
  float *partials;        // [CTAs][partial_slots][partial_floats]
};

__device__ __forceinline__ float exp2_fast(float x) {  // ex2.approx: 2 ulp, exact limits
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

template <int DT>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (DT == MLORA_BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// (x, y) rounded to a pair, and the pair of what the rounding left.
template <int DT>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t &hi, uint32_t &lo) {
  const uint16_t hx = Elem<DT>::from_float(x), hy = Elem<DT>::from_float(y);
  hi = (uint32_t)hx | ((uint32_t)hy << 16);
  lo = (uint32_t)Elem<DT>::from_float(x - Elem<DT>::lo(hx)) |
       ((uint32_t)Elem<DT>::from_float(y - Elem<DT>::lo(hy)) << 16);
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Place in the list of tiles: rows, then heads (key-value head, chunk of its group), then the row's tiles.
struct Cursor {
  int row, hc, tile, ntiles;
  int pos, lo;  // tokens lo .. pos are seen
};

template <int DP, int NW>
struct AttnSmem {
  static constexpr int kStages = attn_stages(DP);
  static constexpr int kStageElems = 2 * kTile * DP;  // K, then V
  uint16_t ring[NW][kStages][kStageElems];
  int64_t first[kRowsPerLaunch + 1];  // tiles (of one head) before a row
  int32_t pos[kRowsPerLaunch];        // last token seen; -1: none, -2: a bad row
  uint32_t seen[NW][kStages];         // bit t: token t of the tile is seen
  int64_t warp_sum[NW];
  int32_t piece_row[NW][2], piece_hc[NW][2];  // a warp's unfinished pieces: [0] without, [1] with the first tile
  int32_t last[2];
};

template <int DT, int DP, bool WIDE>
__global__ void __launch_bounds__(attn_warps(DP) * 32, 1)
    kv_attention_kernel(const __grid_constant__ AttnParams p, int32_t *status) {
  constexpr int NW = attn_warps(DP), NT = NW * 32;
  using Smem = AttnSmem<DP, NW>;
  constexpr int S = Smem::kStages;
  constexpr int CH = DP / 8;         // 16-byte chunks of a token's head
  constexpr int GP = WIDE ? 16 : 8;  // heads that a piece's partial result holds
  constexpr float kShift = DT == MLORA_FP16 ? 15.f : 0.f;  // weights up to 2^15 keep small ones out of fp16's subnormals
  extern __shared__ __align__(128) char smem_raw[];
  Smem &sh = *reinterpret_cast<Smem *>(smem_raw);
  const mlora_kv_attn &a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int D = p.c.head_dim, HC = p.c.num_kv_heads * p.chunks;
  pdl_wait();
  pdl_launch_dependents();

  // ---- the list of tiles: exclusive sums of the rows' tile counts ------------------------------
  const int R = p.rows;
  {
    const int each = (R + NT - 1) / NT;
    int64_t sum = 0;
    int bad = 0;
    for (int i = 0; i < each; ++i) {
      const int r = tid * each + i;
      if (r >= R) break;
      const int64_t row = (int64_t)p.row0 + r;
      int pos = a.position[row], n = 0;
      const int req = a.row_request ? a.row_request[row] : (int)row;
      if (pos < -1 || pos >= (int64_t)a.max_pages * p.page.d) bad |= MLORA_STATUS_BAD_LENGTH, pos = -2;
      else if (pos >= 0 && (req < 0 || req >= a.num_requests)) bad |= MLORA_STATUS_BAD_REQUEST, pos = -2;
      if (pos >= 0) {
        const int lo = a.window ? max(0, pos + 1 - a.window) : 0;
        n = pos / kTile - lo / kTile + 1;
      }
      sh.pos[r] = pos;
      sh.first[r] = n;
      sum += n;
    }
    int64_t incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(~0u, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) sh.warp_sum[warp] = incl;
    if (bad && blockIdx.x == 0) report(status, bad);
    if (tid < 2 * NW) sh.piece_row[tid >> 1][tid & 1] = -1;
    __syncthreads();
    int64_t at = incl - sum;
    for (int w = 0; w < warp; ++w) at += sh.warp_sum[w];
    for (int i = 0; i < each; ++i) {
      const int r = tid * each + i;
      if (r >= R) break;
      const int64_t n = sh.first[r];
      sh.first[r] = at;
      at += n;
    }
    if (tid == NT - 1) sh.first[R] = at;
    __syncthreads();
  }
  // rows that see nothing
  for (int r = blockIdx.x; r < R; r += gridDim.x) {
    if (sh.pos[r] != -1) continue;
    const int64_t row = (int64_t)p.row0 + r;
    uint4 *o = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + row * a.ldo);
    for (int i = tid; i < a.num_q_heads * D / 8; i += NT) o[i] = make_uint4(0, 0, 0, 0);
    if (a.lse)
      for (int i = tid; i < a.num_q_heads; i += NT) a.lse[row * a.num_q_heads + i] = -CUDART_INF_F;
  }

  // ---- this CTA's and this warp's part of it -----------------------------------------------------
  const int64_t T = sh.first[R] * HC;
  const int64_t shares = (T + kMinTiles - 1) / kMinTiles;
  const int C = (int)min((int64_t)gridDim.x, shares);
  if ((int)blockIdx.x >= C) return;
  const int nw = (int)min((int64_t)NW, (shares + C - 1) / C);
  const int64_t t0 = blockIdx.x * T / C, t1 = (blockIdx.x + 1) * T / C;
  const int64_t w0 = t0 + warp * (t1 - t0) / nw, w1 = warp < nw ? t0 + (warp + 1) * (t1 - t0) / nw : w0;
  const int n = (int)(w1 - w0);

  auto set_row = [&](Cursor &c) {
    c.pos = sh.pos[c.row];
    c.lo = a.window ? max(0, c.pos + 1 - a.window) : 0;
    c.ntiles = (int)(sh.first[c.row + 1] - sh.first[c.row]);
  };
  auto next = [&](Cursor &c) {
    if (++c.tile < c.ntiles) return;
    c.tile = 0;
    if (++c.hc < HC) return;
    c.hc = 0;
    do ++c.row;
    while (c.row < R && sh.first[c.row + 1] == sh.first[c.row]);
    if (c.row < R) set_row(c);
  };

  float *const partials = p.partials + (int64_t)blockIdx.x * partial_slots(DP) * partial_floats(DP);
  if (n > 0) {
    Cursor cur;  // of the tile that is computed
    {
      // the last row with first[row] <= w0 / HC: 32 rows a step, two steps
      const int64_t x = w0 / HC;
      const int stride = (R + 31) / 32;
      const int probe = lane * stride;
      const int blk = __popc(__ballot_sync(~0u, probe < R && sh.first[min(probe, R)] <= x)) - 1;
      const int in = blk * stride + lane;
      cur.row = blk * stride +
                __popc(__ballot_sync(~0u, lane < stride && in < R && sh.first[min(in, R)] <= x)) - 1;
      set_row(cur);
      const int64_t rem = w0 - sh.first[cur.row] * HC;
      cur.hc = (int)(rem / cur.ntiles);
      cur.tile = (int)(rem - (int64_t)cur.hc * cur.ntiles);
    }
    Cursor ahead = cur;  // of the tile whose page ids are looked up

    // ---- loads: page ids one tile ahead of the copies, copies S - 1 tiles ahead of the products ------
    int32_t id = -1, inpage = 0;  // lanes 0-15: page and place in it of the tile's token `lane`
    int kv_head = 0;
    bool want = false;
    auto look_up = [&]() {  // the tile at `ahead`
      const int t = (ahead.lo / kTile + ahead.tile) * kTile + (lane & 15);
      want = t >= ahead.lo && t <= ahead.pos;
      const int64_t row = (int64_t)p.row0 + ahead.row;
      const int req = a.row_request ? a.row_request[row] : (int)row;
      const int pg = div_by(p.page, t);
      inpage = t - pg * p.page.d;
      id = want ? a.page_table[(int64_t)req * a.table_stride + pg] : -1;
      kv_head = p.chunks == 1 ? ahead.hc : ahead.hc / p.chunks;
      next(ahead);
    };
    auto issue = [&](int slot) {  // the tile last looked up, into ring slot `slot`
      const bool good = want && id >= 0 && id < p.c.num_pages;
      if (want && !good) report(status, MLORA_STATUS_BAD_PAGE);
      const int64_t off = good ? (int64_t)id * p.c.page_stride + (int64_t)inpage * p.c.token_stride +
                                     (int64_t)kv_head * p.c.head_stride
                               : 0;
      const uint32_t seen = __ballot_sync(~0u, good) & 0xFFFFu;
      if (lane == 0) sh.seen[warp][slot] = seen;
      uint16_t *ks = sh.ring[warp][slot], *vs = ks + kTile * DP;
#pragma unroll
      for (int i = 0; i < kTile * CH / 32; ++i) {
        const int t = (i * 32 + lane) / CH, ch = lane % CH;
        const int64_t o = __shfl_sync(~0u, off, t) + ch * 8;
        const uint32_t bytes = ((seen >> t) & 1u) && ch * 8 < D ? 16u : 0u;
        const int at = t * DP + ((ch ^ (t & 7)) * 8);
        tc::cp_async16(ks + at, p.k + (bytes ? o : 0), bytes);
        tc::cp_async16(vs + at, p.v + (bytes ? o : 0), bytes);
      }
    };
    look_up();
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
      if (i < n) {
        issue(i);
        if (i + 1 < n) look_up();
      }
      cp_async_commit();
    }

    // ---- products ----------------------------------------------------------------------------------
    const int g = lane >> 2, quad = lane & 3;
    uint32_t q[DP / 16][4];
    float o[DP / 8][4];
    float m[2], l[2];
    bool start = true;  // the next tile is the first of a piece
    int from = 0;       // first tile of the current piece
    // lane's row and chunk in ldmatrix, for K (row: token, plain) and V (row: token, transposed)
    const int kt = ((lane >> 4) << 3) + (lane & 7), kc = (lane >> 3) & 1;
    const int vt = (((lane >> 3) & 1) << 3) + (lane & 7), vc = lane >> 4;
    int slot = 0;
    for (int it = 0; it < n; ++it) {
      const int64_t row = (int64_t)p.row0 + cur.row;
      const int hk = p.chunks == 1 ? cur.hc : cur.hc / p.chunks;
      const int g0 = p.chunks == 1 ? 0 : (cur.hc - hk * p.chunks) * kMaxGroup;
      const int gn = min(p.group - g0, kMaxGroup);
      const int64_t head0 = (int64_t)hk * p.group + g0;
      if (start) {
        from = cur.tile;
        const uint16_t *qr = static_cast<const uint16_t *>(a.q) + row * a.ldq + head0 * D;
#pragma unroll
        for (int kk = 0; kk < DP / 16; ++kk)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int head = g + (j & 1) * 8, d = kk * 16 + quad * 2 + (j >> 1) * 8;
            q[kk][j] = (WIDE || !(j & 1)) && head < gn && d < D
                           ? *reinterpret_cast<const uint32_t *>(qr + (int64_t)head * D + d)
                           : 0u;
          }
#pragma unroll
        for (int j = 0; j < DP / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
        m[0] = m[1] = -CUDART_INF_F;
        l[0] = l[1] = 0.f;
        start = false;
      }
      if (it + S - 1 < n) {
        int into = slot + S - 1;
        if (into >= S) into -= S;
        issue(into);
        if (it + S < n) look_up();
      }
      cp_async_commit();
      cp_async_wait<S - 1>();
      __syncwarp();
      const uint32_t seen = sh.seen[warp][slot];
      const uint32_t ks = smem_u32(sh.ring[warp][slot]), vs = ks + kTile * DP * 2;

      float s[2][4] = {};
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk) {
        uint32_t b[4];
        ldmatrix4(b, ks + kt * DP * 2 + (((kk * 2 + kc) ^ (kt & 7)) << 4));
        mma<DT>(s[0], q[kk], b[0], b[1]);
        mma<DT>(s[1], q[kk], b[2], b[3]);
      }
      // s[nb][0..1]: head g, tokens nb * 8 + quad * 2 + {0, 1}; s[nb][2..3]: head g + 8
#pragma unroll
      for (int nb = 0; nb < 2; ++nb)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          s[nb][j] = (seen >> (nb * 8 + quad * 2 + (j & 1))) & 1u ? s[nb][j] * p.scale_log2 : -CUDART_INF_F;
      float keep[2] = {1.f, 1.f}, base[2];
      bool grew = false;
#pragma unroll
      for (int h = 0; h < (WIDE ? 2 : 1); ++h) {
        float top = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
        if (top > m[h]) {
          keep[h] = exp2_fast(m[h] - top);
          m[h] = top;
          grew = true;
        }
        base[h] = m[h] == -CUDART_INF_F ? 0.f : m[h] - kShift;
      }
      if (!WIDE) keep[1] = keep[0];
      if (__any_sync(~0u, grew)) {
        l[0] *= keep[0];
        if (WIDE) l[1] *= keep[1];
#pragma unroll
        for (int j = 0; j < DP / 8; ++j) {
          o[j][0] *= keep[0], o[j][1] *= keep[0];
          o[j][2] *= keep[1], o[j][3] *= keep[1];
        }
      }
      uint32_t hi[4], lo[4];  // the second product's A: weights, and what their rounding left
#pragma unroll
      for (int nb = 0; nb < 2; ++nb)
#pragma unroll
        for (int h = 0; h < (WIDE ? 2 : 1); ++h) {
          const float x = exp2_fast(s[nb][2 * h] - base[h]), y = exp2_fast(s[nb][2 * h + 1] - base[h]);
          l[h] += x + y;
          split_pair<DT>(x, y, hi[nb * 2 + h], lo[nb * 2 + h]);
        }
      if (!WIDE) hi[1] = lo[0], hi[3] = lo[2];
#pragma unroll
      for (int nn = 0; nn < DP / 16; ++nn) {
        uint32_t b[4];
        ldmatrix4_t(b, vs + vt * DP * 2 + (((nn * 2 + vc) ^ (vt & 7)) << 4));
        mma<DT>(o[2 * nn], hi, b[0], b[1]);
        mma<DT>(o[2 * nn + 1], hi, b[2], b[3]);
        if (WIDE) {
          mma<DT>(o[2 * nn], lo, b[0], b[1]);
          mma<DT>(o[2 * nn + 1], lo, b[2], b[3]);
        }
      }
      __syncwarp();  // the slot may be filled again
      if (++slot == S) slot = 0;

      const bool ends = cur.tile == cur.ntiles - 1;
      if (ends || it == n - 1) {  // the piece is done
        start = true;
#pragma unroll
        for (int h = 0; h < (WIDE ? 2 : 1); ++h) {
          l[h] += __shfl_xor_sync(~0u, l[h], 1);
          l[h] += __shfl_xor_sync(~0u, l[h], 2);
        }
        if (!WIDE)
#pragma unroll
          for (int j = 0; j < DP / 8; ++j) o[j][0] += o[j][2], o[j][1] += o[j][3];
        if (ends && from == 0) {
#pragma unroll
          for (int h = 0; h < (WIDE ? 2 : 1); ++h) {
            const int head = g + 8 * h;
            if (head >= gn) continue;
            const float inv = l[h] == 0.f ? 0.f : 1.f / l[h];
            uint16_t *dst = static_cast<uint16_t *>(a.out) + row * a.ldo + (head0 + head) * D;
#pragma unroll
            for (int j = 0; j < DP / 8; ++j)
              if (j * 8 < D)
                *reinterpret_cast<uint32_t *>(dst + j * 8 + quad * 2) =
                    (uint32_t)Elem<DT>::from_float(o[j][2 * h] * inv) |
                    ((uint32_t)Elem<DT>::from_float(o[j][2 * h + 1] * inv) << 16);
            if (a.lse && quad == 0)
              a.lse[row * a.num_q_heads + head0 + head] =
                  l[h] == 0.f ? -CUDART_INF_F : (m[h] - kShift) * CUDART_LN2_F + logf(l[h]);
          }
        } else {
          const int which = from == 0 ? 1 : 0;
          float *part = partials + (warp * 2 + which) * partial_floats(DP);
#pragma unroll
          for (int h = 0; h < (WIDE ? 2 : 1); ++h) {
            const int head = g + 8 * h;
#pragma unroll
            for (int j = 0; j < DP / 8; ++j)
              *reinterpret_cast<float2 *>(part + head * DP + j * 8 + quad * 2) = make_float2(o[j][2 * h], o[j][2 * h + 1]);
            if (quad == 0) part[kMaxGroup * DP + head] = m[h], part[kMaxGroup * DP + 16 + head] = l[h];
          }
          if (lane == 0) sh.piece_row[warp][which] = cur.row, sh.piece_hc[warp][which] = cur.hc;
        }
      }
      next(cur);
    }
  }
  cp_async_wait<0>();
  __syncthreads();

  // ---- join the pieces of the CTA's warps, then those of the CTAs ------------------------------------
  // `count` partial results, the i-th at at(i), into the output (done) or into partial result `to`.
  auto join = [&](int count, auto at, int r, int hc, bool done, float *to) {
    const int hk = hc / p.chunks, g0 = (hc - hk * p.chunks) * kMaxGroup, gn = min(p.group - g0, kMaxGroup);
    const int64_t row = (int64_t)p.row0 + r, head0 = (int64_t)hk * p.group + g0;
    for (int i = tid; i < GP * (DP / 4); i += NT) {
      const int head = i / (DP / 4), d = (i % (DP / 4)) * 4;
      if (head >= gn) continue;
      float top = -CUDART_INF_F;
      for (int e = 0; e < count; ++e) top = fmaxf(top, __ldcg(at(e) + kMaxGroup * DP + head));
      const float base = top == -CUDART_INF_F ? 0.f : top;
      float sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int e = 0; e < count; ++e) {
        const float *x = at(e);
        const float w = exp2_fast(__ldcg(x + kMaxGroup * DP + head) - base);
        const float4 f = __ldcg(reinterpret_cast<const float4 *>(x + head * DP + d));
        sum += w * __ldcg(x + kMaxGroup * DP + 16 + head);
        acc.x += w * f.x, acc.y += w * f.y, acc.z += w * f.z, acc.w += w * f.w;
      }
      if (done) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        if (d < D) {
          uint2 u;
          u.x = (uint32_t)Elem<DT>::from_float(acc.x * inv) | ((uint32_t)Elem<DT>::from_float(acc.y * inv) << 16);
          u.y = (uint32_t)Elem<DT>::from_float(acc.z * inv) | ((uint32_t)Elem<DT>::from_float(acc.w * inv) << 16);
          *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + row * a.ldo + (head0 + head) * D + d) = u;
        }
        if (a.lse && d == 0)
          a.lse[row * a.num_q_heads + head0 + head] =
              sum == 0.f ? -CUDART_INF_F : (top - kShift) * CUDART_LN2_F + logf(sum);
      } else {
        *reinterpret_cast<float4 *>(to + head * DP + d) = acc;
        if (d == 0) to[kMaxGroup * DP + head] = top, to[kMaxGroup * DP + 16 + head] = sum;
      }
    }
  };
  // Runs of pieces of one (row, head), in the order of the list. The first may have begun in an earlier CTA
  // (it goes to the CTA's partial result 0), the last may go on in a later one (1).
  int open_row[2] = {-1, -1}, open_hc[2] = {0, 0};
  for (int e = 0; e < 2 * nw;) {
    const int r = sh.piece_row[e >> 1][e & 1], hc = sh.piece_hc[e >> 1][e & 1];
    if (r < 0) {
      ++e;
      continue;
    }
    int idx[2 * NW], count = 0;  // entries of the run
    for (; e < 2 * nw; ++e) {
      const int r2 = sh.piece_row[e >> 1][e & 1];
      if (r2 < 0) continue;
      if (r2 != r || sh.piece_hc[e >> 1][e & 1] != hc) break;
      idx[count++] = e;
    }
    const int64_t nt = sh.first[r + 1] - sh.first[r], begin = sh.first[r] * HC + hc * nt;
    const bool here = begin >= t0, done = here && begin + nt <= t1;
    if (!done) open_row[here] = r, open_hc[here] = hc;
    join(count, [&](int i) { return partials + idx[i] * partial_floats(DP); }, r, hc, done,
         partials + (2 * NW + (here ? 1 : 0)) * partial_floats(DP));
  }
  if (open_row[0] < 0 && open_row[1] < 0) return;
  __threadfence();
  __syncthreads();
  int64_t c0[2], c1[2];  // first and last CTA of the open items
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (open_row[h] < 0) continue;
    const int64_t nt = sh.first[open_row[h] + 1] - sh.first[open_row[h]];
    const int64_t begin = sh.first[open_row[h]] * HC + open_hc[h] * nt;
    c0[h] = ((begin + 1) * C - 1) / T;
    c1[h] = ((begin + nt) * C - 1) / T;
    if (tid == 0) {
      const int before = atomicAdd(p.counters + c0[h], 1);
      sh.last[h] = before == (int)(c1[h] - c0[h]);
      if (sh.last[h]) p.counters[c0[h]] = 0;  // nobody else comes: back to zero for the next call
    }
  }
  if (tid == 0) __threadfence();
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (open_row[h] < 0 || !sh.last[h]) continue;
    const int64_t first = c0[h];
    join((int)(c1[h] - first + 1),
         [&](int i) {
           return p.partials + ((first + i) * partial_slots(DP) + 2 * NW + (i == 0 ? 1 : 0)) * partial_floats(DP);
         },
         open_row[h], open_hc[h], true, nullptr);
  }
}

int attn_ctas() { return sm_count(); }
constexpr size_t kCounterBytes = 4096;  // more than any GPU's SMs

template <int DT, int DP, bool WIDE>
cudaError_t launch(const AttnParams &p, int32_t *status, cudaStream_t stream) {
  using Smem = AttnSmem<DP, attn_warps(DP)>;
  static_assert(sizeof(Smem) <= 227 * 1024, "fits in shared memory");
  cudaError_t e = cudaFuncSetAttribute(kv_attention_kernel<DT, DP, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)sizeof(Smem));
  if (e != cudaSuccess) return e;
  e = launch_waiting(kv_attention_kernel<DT, DP, WIDE>, dim3(attn_ctas()), dim3(attn_warps(DP) * 32), sizeof(Smem), 1,
                     stream, p, status);
  if (e == cudaSuccess) api_count_launch();
  return e;
}

template <int DT>
cudaError_t dispatch(const AttnParams &p, int32_t *status, cudaStream_t stream) {
  const bool wide = p.group > 8;
  switch (padded_dim(p.c.head_dim)) {
    case 64: return wide ? launch<DT, 64, true>(p, status, stream) : launch<DT, 64, false>(p, status, stream);
    case 128: return wide ? launch<DT, 128, true>(p, status, stream) : launch<DT, 128, false>(p, status, stream);
    default: return wide ? launch<DT, 256, true>(p, status, stream) : launch<DT, 256, false>(p, status, stream);
  }
}

}  // namespace

int64_t kv_attention_workspace_bytes(int32_t head_dim) {
  const int dp = padded_dim(head_dim);
  return (int64_t)kCounterBytes + (int64_t)attn_ctas() * partial_slots(dp) * partial_floats(dp) * sizeof(float);
}

cudaError_t launch_kv_attention(const mlora_kv_cache &c, const mlora_kv_attn &a, int32_t layer, int32_t *status,
                                cudaStream_t stream) {
  AttnParams p{};
  p.c = c;
  p.a = a;
  p.k = static_cast<const uint16_t *>(c.k) + layer * c.layer_stride;
  p.v = static_cast<const uint16_t *>(c.v) + layer * c.layer_stride;
  p.page = fast_div(c.page_tokens);
  p.group = a.num_q_heads / c.num_kv_heads;
  p.chunks = (p.group + kMaxGroup - 1) / kMaxGroup;
  p.scale_log2 = a.scale * 1.44269504088896340736f;
  p.counters = static_cast<int32_t *>(a.workspace);
  p.partials = reinterpret_cast<float *>(static_cast<char *>(a.workspace) + kCounterBytes);
  for (int32_t row0 = 0; row0 < a.num_rows; row0 += kRowsPerLaunch) {
    p.row0 = row0;
    p.rows = min(kRowsPerLaunch, a.num_rows - row0);
    const cudaError_t e = c.dtype == MLORA_BF16 ? dispatch<MLORA_BF16>(p, status, stream)
                                                : dispatch<MLORA_FP16>(p, status, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace mlora
