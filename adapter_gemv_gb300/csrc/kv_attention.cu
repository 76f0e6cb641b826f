// kv_attention.cu -- attention of new tokens over the paged key-value cache (sm_103a).
//
//   s_t = scale q.K_t,  m = max_t s_t,  l = sum_t exp(s_t - m),  out = sum_t exp(s_t - m) V_t / l
// in one pass over the tokens, with a running m, and l and out rescaled by exp(m - m') when it moves.
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
//     next without draining its ring. Every 32 tiles its lanes work out 32 tiles' places at once.
//   * A (row, head) cut between warps is joined in two steps, in a fixed order: the warps of a CTA, in
//     shared memory, then the CTAs, by the one that finishes last (a counter that it returns to zero).
// What a warp does between two tiles has to stay below the time its share of the bandwidth gives it
// (some 2800 cycles at 8 KB a tile and 8 warps), with room to catch up, so the instructions are few:
//   * Products transposed, S^T = K Q^T and O^T = V^T P^T: tokens (then head elements) are the 16 rows of
//     m16n8k16 and the group's heads its 8 columns, of which a group of 8 fills all. (With the heads
//     as rows, half of every product is padding, and the accumulators twice as many.)
//   * The maximum is not followed exactly: m moves when a score passes it by 2^kSlack, which one vote
//     per tile decides; weights up to 2^kSlack are as exact as those up to 1.
//   * The weights are rounded to 16 bits for the second product. Their remainder, rounded likewise, goes
//     through a second one, so what is left is fp32's error; the products cost nothing (above).
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "serve.cuh"
#include "tc.cuh"

namespace mlora {

namespace {

constexpr int kTile = 16;            // tokens of a tile
constexpr int kRowsPerLaunch = 1024;
constexpr int kMinTiles = 4;         // a warp's share of a small call, so that few pieces have to be joined
constexpr int kMaxGroup = 16;        // query heads of a work item
constexpr float kSlack = 8.f;        // log2 of how far a weight may pass 1 before m moves

constexpr int attn_warps(int dp) { return dp == 256 ? 4 : 8; }
constexpr int attn_stages(int dp) { return dp == 64 ? 6 : 3; }
// Floats of a partial result: out [16][dp], then m [16] and l [16].
constexpr int partial_floats(int dp) { return kMaxGroup * (dp + 2); }
// Partial results of a CTA in the workspace: one a warp, two of its own.
constexpr int partial_slots(int dp) { return attn_warps(dp) + 2; }
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
// Transpose of an 8 x 8 matrix of 16-bit elements held a row per four lanes.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
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

// A tile's place, one per lane for 32 consecutive tiles of the list.
struct Tile {
  int64_t off;    // pages of whole tiles: its first token in the cache; else its request and first token
  uint32_t seen;  // bit t: token t is seen
  uint32_t row;   // the row, with kFirst / kLast for the first / last tile of its (row, head)
  int32_t hc;     // key-value head and chunk of its group
};
constexpr uint32_t kFirst = 1u << 30, kLast = 1u << 31, kRowMask = kFirst - 1;

template <int DP, int NW>
struct AttnSmem {
  static constexpr int kStages = attn_stages(DP);
  static constexpr int kStageElems = 2 * kTile * DP;  // K, then V
  // a warp's tiles; after its last tile, its two unfinished pieces [2][16][DP] fp32
  uint16_t ring[NW][kStages][kStageElems];
  int64_t first[kRowsPerLaunch + 1];  // tiles (of one head) before a row
  int32_t pos[kRowsPerLaunch];        // last token seen; -1: none, -2: a bad row
  uint32_t seen[NW][kStages];         // bit t: token t of the tile is seen
  int64_t warp_sum[NW];
  float m[2 * NW][kMaxGroup], l[2 * NW][kMaxGroup];  // of the pieces: [2w] without the first tile, [2w+1] with it
  int32_t piece_row[2 * NW], piece_hc[2 * NW];
  int32_t run[2 * NW + 1], runs;  // where the joined pieces of one (row, head) start, in order[]
  int32_t order[2 * NW];
  int32_t last[2];
};

// PAGED16: a page holds whole tiles. NB: blocks of 8 heads of a group's chunk.
template <int DT, int DP, int NB, bool PAGED16>
__global__ void __launch_bounds__(attn_warps(DP) * 32, 1)
    kv_attention_kernel(const __grid_constant__ AttnParams p, int32_t *status) {
  constexpr int NW = attn_warps(DP), NT = NW * 32;
  using Smem = AttnSmem<DP, NW>;
  constexpr int S = Smem::kStages;
  constexpr int CH = DP / 8;    // 16-byte chunks of a token's head
  constexpr int GP = NB * 8;    // heads that a piece holds
  static_assert(2 * GP * DP * 4 <= S * Smem::kStageElems * 2, "the pieces fit in the ring");
  // fp16 weights: up to 2^15 (with kSlack), so that small ones stay out of fp16's subnormals
  constexpr float kShift = DT == MLORA_FP16 ? 7.f : 0.f;
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
    if (tid < 2 * NW) sh.piece_row[tid] = -1;
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

  float *const partials = p.partials + (int64_t)blockIdx.x * partial_slots(DP) * partial_floats(DP);
  // chunks past the head's end are never copied: zero for good
  if (D < DP) {
    for (int i = lane; i < S * Smem::kStageElems / 8; i += 32)
      reinterpret_cast<uint4 *>(sh.ring[warp])[i] = make_uint4(0, 0, 0, 0);
    __syncwarp();
  }
  if (n > 0) {
    // tiles w0 + 32 b + lane
    auto place = [&](int b) {
      Tile t{};
      const int64_t x = w0 + (int64_t)b * 32 + lane;
      if (x >= w1) return t;
      int r = 0;
      for (int hi = R; hi - r > 1;) {  // the last row with first[row] HC <= x
        const int mid = (r + hi) >> 1;
        if (sh.first[mid] * HC <= x) r = mid;
        else hi = mid;
      }
      const int nt = (int)(sh.first[r + 1] - sh.first[r]);
      const int64_t rem = x - sh.first[r] * HC;
      t.hc = rem < nt ? 0 : (int)(rem / nt);
      const int tile = (int)(rem - (int64_t)t.hc * nt);
      const int pos = sh.pos[r], lo = a.window ? max(0, pos + 1 - a.window) : 0;
      const int t0 = (lo / kTile + tile) * kTile;
      t.seen = 0xFFFFu;
      if (t0 < lo) t.seen &= 0xFFFFu << (lo - t0);
      if (pos - t0 < kTile - 1) t.seen &= (2u << (pos - t0)) - 1u;
      t.row = (uint32_t)r | (tile == 0 ? kFirst : 0u) | (tile == nt - 1 ? kLast : 0u);
      const int64_t row = (int64_t)p.row0 + r;
      const int req = a.row_request ? a.row_request[row] : (int)row;
      if constexpr (PAGED16) {
        const int pg = div_by(p.page, t0);
        const int id = a.page_table[(int64_t)req * a.table_stride + pg];
        if (id >= 0 && id < p.c.num_pages) {
          t.off = (int64_t)id * p.c.page_stride + (int64_t)(t0 - pg * p.page.d) * p.c.token_stride +
                  (int64_t)(p.chunks == 1 ? t.hc : t.hc / p.chunks) * p.c.head_stride;
        } else {
          report(status, MLORA_STATUS_BAD_PAGE);
          t.seen = 0;
        }
      } else {
        t.off = ((int64_t)req << 32) | (uint32_t)t0;
      }
      return t;
    };
    Tile cur = place(0), nxt{};
    if (n > 32) nxt = place(1);
    int cur_batch = 0;

    // ---- loads, S - 1 tiles ahead of the products --------------------------------------------------
    const int lt = lane / CH, lc = lane % CH;  // a lane's token and chunk within a step of 32 chunks
    constexpr int kStep = 32 / CH;             // tokens of such a step
    const bool mine = lc * 8 < D;
    // pages of other sizes: each token's page, looked up a tile before its copies start
    int id = -1, inpage = 0, kv_head = 0;
    uint32_t range = 0;
    auto look_up = [&](int i) {
      const Tile &b = (i >> 5) == cur_batch ? cur : nxt;
      const int64_t at = __shfl_sync(~0u, b.off, i & 31);
      const int hc = __shfl_sync(~0u, b.hc, i & 31);
      range = __shfl_sync(~0u, b.seen, i & 31);
      const int t = (int)(uint32_t)at + (lane & 15), pg = div_by(p.page, t);
      inpage = t - pg * p.page.d;
      id = (range >> (lane & 15)) & 1u ? a.page_table[(at >> 32) * a.table_stride + pg] : -1;
      kv_head = p.chunks == 1 ? hc : hc / p.chunks;
    };
    auto issue = [&](int i, int slot) {  // tile i into ring slot `slot`
      uint16_t *ks = sh.ring[warp][slot];
      if constexpr (PAGED16) {
        const Tile &b = (i >> 5) == cur_batch ? cur : nxt;
        const int64_t off = __shfl_sync(~0u, b.off, i & 31);
        const uint32_t seen = __shfl_sync(~0u, b.seen, i & 31);
        if (lane == 0) sh.seen[warp][slot] = seen;
        if (mine) {
          const int64_t at = off + (int64_t)lt * p.c.token_stride + lc * 8;
          const uint16_t *pk = p.k + at, *pv = p.v + at;
          const int64_t step = kStep * p.c.token_stride;
#pragma unroll
          for (int j = 0; j < kTile / kStep; ++j) {
            const int t = j * kStep + lt;
            uint16_t *dst = ks + t * DP + ((lc ^ (t & 7)) * 8);
            const uint32_t bytes = (seen >> t) & 1u ? 16u : 0u;
            tc::cp_async16(dst, bytes ? pk : p.k, bytes);
            tc::cp_async16(dst + kTile * DP, bytes ? pv : p.v, bytes);
            pk += step, pv += step;
          }
        }
      } else {
        const bool want = (range >> (lane & 15)) & 1u, good = want && id >= 0 && id < p.c.num_pages;
        if (want && !good) report(status, MLORA_STATUS_BAD_PAGE);
        const int64_t off = good ? (int64_t)id * p.c.page_stride + (int64_t)inpage * p.c.token_stride +
                                       (int64_t)kv_head * p.c.head_stride
                                 : 0;
        const uint32_t seen = __ballot_sync(~0u, good) & 0xFFFFu;
        if (lane == 0) sh.seen[warp][slot] = seen;
#pragma unroll
        for (int j = 0; j < kTile / kStep; ++j) {
          const int t = j * kStep + lt;
          const int64_t o = __shfl_sync(~0u, off, t) + lc * 8;
          const uint32_t bytes = (seen >> t) & 1u ? 16u : 0u;
          uint16_t *dst = ks + t * DP + ((lc ^ (t & 7)) * 8);
          if (mine) {
            tc::cp_async16(dst, p.k + (bytes ? o : 0), bytes);
            tc::cp_async16(dst + kTile * DP, p.v + (bytes ? o : 0), bytes);
          }
        }
        if (i + 1 < n) look_up(i + 1);
      }
    };
    if constexpr (!PAGED16) look_up(0);
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
      if (i < n) issue(i, i);
      cp_async_commit();
    }

    // ---- products ----------------------------------------------------------------------------------
    const int g = lane >> 2, quad = lane & 3;
    uint32_t q[DP / 16][NB][2];  // Q^T: head elements kk * 16 + {0, 8} + quad * 2 + {0, 1}, head g of the block
    float o[DP / 16][NB][4];     // O^T: elements j * 16 + g (0, 1) and + 8 (2, 3), heads quad * 2 + {0, 1}
    float m[NB][2], l[NB][2];    // of heads quad * 2 + {0, 1}; l: of this lane's tokens
    bool start = true, with_first = false;
    int row_in = 0, hc = 0, gn = 0;
    int64_t row = 0, head0 = 0;
    // lane's row and chunk in ldmatrix: K (token, plain) and V (token, transposed)
    const int kt = lane & 15, kc = lane >> 4;
    const int vt = (lane & 7) + ((lane >> 4) << 3), vc = (lane >> 3) & 1;
    int slot = 0;
    for (int it = 0; it < n; ++it) {
      if ((it & 31) == 0 && it) {
        cur = nxt;
        ++cur_batch;
        if (it + 32 < n) nxt = place(cur_batch + 1);
      }
      const uint32_t meta = __shfl_sync(~0u, cur.row, it & 31);
      if (start) {
        row_in = (int)(meta & kRowMask);
        hc = __shfl_sync(~0u, cur.hc, it & 31);
        with_first = (meta & kFirst) != 0;
        row = (int64_t)p.row0 + row_in;
        const int hk = p.chunks == 1 ? hc : hc / p.chunks;
        const int g0 = p.chunks == 1 ? 0 : (hc - hk * p.chunks) * kMaxGroup;
        gn = min(p.group - g0, kMaxGroup);
        head0 = (int64_t)hk * p.group + g0;
        const uint16_t *qr = static_cast<const uint16_t *>(a.q) + row * a.ldq + head0 * D;
#pragma unroll
        for (int kk = 0; kk < DP / 16; ++kk)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int head = nb * 8 + g, d = kk * 16 + j * 8 + quad * 2;
              q[kk][nb][j] =
                  head < gn && d < D ? *reinterpret_cast<const uint32_t *>(qr + (int64_t)head * D + d) : 0u;
            }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
          for (int j = 0; j < DP / 16; ++j) o[j][nb][0] = o[j][nb][1] = o[j][nb][2] = o[j][nb][3] = 0.f;
          m[nb][0] = m[nb][1] = -CUDART_INF_F;
          l[nb][0] = l[nb][1] = 0.f;
        }
        start = false;
      }
      if (it + S - 1 < n) issue(it + S - 1, slot == 0 ? S - 1 : slot - 1);
      cp_async_commit();
      cp_async_wait<S - 1>();
      __syncwarp();
      const uint32_t seen = sh.seen[warp][slot];
      const uint32_t ks = smem_u32(sh.ring[warp][slot]), vs = ks + kTile * DP * 2;

      float s[NB][4] = {}, s2[NB][4] = {};  // two chains of products
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk) {
        uint32_t x[4];
        ldmatrix4(x, ks + kt * DP * 2 + (((kk * 2 + kc) ^ (kt & 7)) << 4));
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) mma<DT>(kk & 1 ? s2[nb] : s[nb], x, q[kk][nb][0], q[kk][nb][1]);
      }
      // s[nb][2 i + j]: token g + 8 i, head quad * 2 + j
      const bool on[2] = {((seen >> g) & 1u) != 0, ((seen >> (g + 8)) & 1u) != 0};
      bool past = false;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[nb][j] = on[j >> 1] ? (s[nb][j] + s2[nb][j]) * p.scale_log2 : -CUDART_INF_F;
          past |= s[nb][j] > m[nb][j & 1] + kSlack;
        }
      if (__any_sync(~0u, past)) {  // m moves to the maximum
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float top = fmaxf(s[nb][j], s[nb][j + 2]);
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 4));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 8));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 16));
            if (top > m[nb][j]) {
              const float keep = exp2_fast(m[nb][j] - top);
              m[nb][j] = top;
              l[nb][j] *= keep;
#pragma unroll
              for (int i = 0; i < DP / 16; ++i) o[i][nb][j] *= keep, o[i][nb][j + 2] *= keep;
            }
          }
      }
      uint32_t hi[NB][2], lo[NB][2];  // P^T: tokens {0, 8} + quad * 2 + {0, 1}, head g
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float base = m[nb][j & 1] == -CUDART_INF_F ? 0.f : m[nb][j & 1] - kShift;
          w[j] = exp2_fast(s[nb][j] - base);
          l[nb][j & 1] += w[j];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t h, r;
          split_pair<DT>(w[2 * i], w[2 * i + 1], h, r);
          hi[nb][i] = transpose8(h);
          lo[nb][i] = transpose8(r);
        }
      }
#pragma unroll
      for (int j = 0; j < DP / 16; ++j) {
        uint32_t x[4];
        ldmatrix4_t(x, vs + vt * DP * 2 + (((j * 2 + vc) ^ (vt & 7)) << 4));
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          mma<DT>(o[j][nb], x, hi[nb][0], hi[nb][1]);
          mma<DT>(o[j][nb], x, lo[nb][0], lo[nb][1]);
        }
      }
      __syncwarp();  // the slot may be filled again
      if (++slot == S) slot = 0;

      if ((meta & kLast) || it == n - 1) {  // the piece is done
        start = true;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            l[nb][j] += __shfl_xor_sync(~0u, l[nb][j], 4);
            l[nb][j] += __shfl_xor_sync(~0u, l[nb][j], 8);
            l[nb][j] += __shfl_xor_sync(~0u, l[nb][j], 16);
          }
        if ((meta & kLast) && with_first) {  // and whole
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int head = nb * 8 + quad * 2 + j;
              if (head >= gn) continue;
              const float inv = l[nb][j] == 0.f ? 0.f : 1.f / l[nb][j];
              uint16_t *dst = static_cast<uint16_t *>(a.out) + row * a.ldo + (head0 + head) * D;
#pragma unroll
              for (int i = 0; i < DP / 16; ++i) {
                if (i * 16 < D) dst[i * 16 + g] = Elem<DT>::from_float(o[i][nb][j] * inv);
                if (i * 16 + 8 < D) dst[i * 16 + 8 + g] = Elem<DT>::from_float(o[i][nb][j + 2] * inv);
              }
              if (a.lse && g == 0)
                a.lse[row * a.num_q_heads + head0 + head] =
                    l[nb][j] == 0.f ? -CUDART_INF_F : (m[nb][j] - kShift) * CUDART_LN2_F + logf(l[nb][j]);
            }
        } else {
          // a piece: at the end of the warp's tiles into its (then idle) ring, before that to the workspace
          const int piece = 2 * warp + (with_first ? 1 : 0);
          float *part = it == n - 1 ? reinterpret_cast<float *>(sh.ring[warp]) + (piece & 1) * GP * DP
                                    : partials + warp * partial_floats(DP);
          if (it == n - 1) {
            cp_async_wait<0>();
            __syncwarp();
          }
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int head = nb * 8 + quad * 2 + j;
              if (head >= gn) continue;
#pragma unroll
              for (int i = 0; i < DP / 16; ++i) {
                part[head * DP + i * 16 + g] = o[i][nb][j];
                part[head * DP + i * 16 + 8 + g] = o[i][nb][j + 2];
              }
              if (g == 0) sh.m[piece][head] = m[nb][j], sh.l[piece][head] = l[nb][j];
            }
          if (lane == 0) {
            sh.piece_row[piece] = row_in;
            sh.piece_hc[piece] = hc | (it == n - 1 ? 0 : 1 << 30);  // bit 30: in the workspace
          }
        }
      }
    }
    // a piece that went to the workspace comes back beside the other
    cp_async_wait<0>();
    __syncwarp();
    if (sh.piece_row[2 * warp] >= 0 && (sh.piece_hc[2 * warp] >> 30)) {
      const float *part = partials + warp * partial_floats(DP);
      const int c = sh.piece_hc[2 * warp] & ~(1 << 30);
      const int heads = min(p.group - (c % p.chunks) * kMaxGroup, kMaxGroup);
      for (int i = lane; i < heads * DP / 4; i += 32)
        reinterpret_cast<float4 *>(sh.ring[warp])[i] = __ldcg(reinterpret_cast<const float4 *>(part) + i);
      __syncwarp();
      if (lane == 0) sh.piece_hc[2 * warp] = c;
    }
  }
  __syncthreads();

  // ---- join the pieces of the CTA's warps, then those of the CTAs ------------------------------------
  if (tid == 0) {  // runs of pieces of one (row, head), in the order of the list
    int runs = 0, count = 0;
    for (int e = 0; e < 2 * nw; ++e) {
      if (sh.piece_row[e] < 0) continue;
      const int before = count ? sh.order[count - 1] : -1;
      if (before < 0 || sh.piece_row[before] != sh.piece_row[e] || sh.piece_hc[before] != sh.piece_hc[e])
        sh.run[runs++] = count;
      sh.order[count++] = e;
    }
    sh.run[runs] = count;
    sh.runs = runs;
  }
  __syncthreads();
  // The first run may have begun in an earlier CTA (it goes to the CTA's partial result 0), the last may go
  // on in a later one (1).
  int open_row[2] = {-1, -1}, open_hc[2] = {0, 0};
  auto emit = [&](int64_t row, int64_t head, int d, float4 acc, float top, float sum) {
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    if (d < D) {
      uint2 u;
      u.x = (uint32_t)Elem<DT>::from_float(acc.x * inv) | ((uint32_t)Elem<DT>::from_float(acc.y * inv) << 16);
      u.y = (uint32_t)Elem<DT>::from_float(acc.z * inv) | ((uint32_t)Elem<DT>::from_float(acc.w * inv) << 16);
      *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + row * a.ldo + head * D + d) = u;
    }
    if (a.lse && d == 0)
      a.lse[row * a.num_q_heads + head] = sum == 0.f ? -CUDART_INF_F : (top - kShift) * CUDART_LN2_F + logf(sum);
  };
  constexpr int kUnits = GP * (DP / 4);  // four elements of a head
  const int runs = sh.runs;
  for (int u = 0; u < runs; ++u) {
    const int e0 = sh.order[sh.run[u]], r = sh.piece_row[e0], c = sh.piece_hc[e0];
    const int64_t nt = sh.first[r + 1] - sh.first[r], begin = sh.first[r] * HC + c * nt;
    const bool here = begin >= t0, done = here && begin + nt <= t1;
    if (!done) open_row[here] = r, open_hc[here] = c;
    const int hk = c / p.chunks, g0 = (c - hk * p.chunks) * kMaxGroup, heads = min(p.group - g0, kMaxGroup);
    float *to = partials + (NW + (here ? 1 : 0)) * partial_floats(DP);
    for (int i = tid; i < kUnits; i += NT) {
      const int head = i / (DP / 4), d = (i % (DP / 4)) * 4;
      if (head >= heads) break;
      float top = -CUDART_INF_F, sum = 0.f;
      for (int k = sh.run[u]; k < sh.run[u + 1]; ++k) top = fmaxf(top, sh.m[sh.order[k]][head]);
      const float base = top == -CUDART_INF_F ? 0.f : top;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k = sh.run[u]; k < sh.run[u + 1]; ++k) {
        const int e = sh.order[k];
        const float w = exp2_fast(sh.m[e][head] - base);
        const float4 f = reinterpret_cast<const float4 *>(sh.ring[e >> 1])[(e & 1) * kUnits + i];
        sum += w * sh.l[e][head];
        acc.x += w * f.x, acc.y += w * f.y, acc.z += w * f.z, acc.w += w * f.w;
      }
      if (done) {
        emit((int64_t)p.row0 + r, (int64_t)hk * p.group + g0 + head, d, acc, top, sum);
      } else {
        *reinterpret_cast<float4 *>(to + head * DP + d) = acc;
        if (d == 0) to[kMaxGroup * DP + head] = top, to[kMaxGroup * DP + 16 + head] = sum;
      }
    }
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
    const int count = (int)(c1[h] - c0[h] + 1), c = open_hc[h];
    const int hk = c / p.chunks, g0 = (c - hk * p.chunks) * kMaxGroup, heads = min(p.group - g0, kMaxGroup);
    auto at = [&](int k) {
      return p.partials + ((c0[h] + k) * partial_slots(DP) + NW + (k == 0 ? 1 : 0)) * partial_floats(DP);
    };
    for (int i = tid; i < kUnits; i += NT) {
      const int head = i / (DP / 4), d = (i % (DP / 4)) * 4;
      if (head >= heads) break;
      float top = -CUDART_INF_F, sum = 0.f;
#pragma unroll 8
      for (int k = 0; k < count; ++k) top = fmaxf(top, __ldcg(at(k) + kMaxGroup * DP + head));
      const float base = top == -CUDART_INF_F ? 0.f : top;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
      for (int k = 0; k < count; ++k) {
        const float *x = at(k);
        const float4 f = __ldcg(reinterpret_cast<const float4 *>(x + head * DP + d));
        const float w = exp2_fast(__ldcg(x + kMaxGroup * DP + head) - base);
        sum += w * __ldcg(x + kMaxGroup * DP + 16 + head);
        acc.x += w * f.x, acc.y += w * f.y, acc.z += w * f.z, acc.w += w * f.w;
      }
      emit((int64_t)p.row0 + open_row[h], (int64_t)hk * p.group + g0 + head, d, acc, top, sum);
    }
  }
}

int attn_ctas() { return sm_count(); }
constexpr size_t kCounterBytes = 4096;  // more than any GPU's SMs

template <int DT, int DP, int NB, bool PAGED16>
cudaError_t launch(const AttnParams &p, int32_t *status, cudaStream_t stream) {
  using Smem = AttnSmem<DP, attn_warps(DP)>;
  static_assert(sizeof(Smem) <= 227 * 1024, "fits in shared memory");
  cudaError_t e = cudaFuncSetAttribute(kv_attention_kernel<DT, DP, NB, PAGED16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)sizeof(Smem));
  if (e != cudaSuccess) return e;
  e = launch_waiting(kv_attention_kernel<DT, DP, NB, PAGED16>, dim3(attn_ctas()), dim3(attn_warps(DP) * 32), sizeof(Smem), 1,
                     stream, p, status);
  if (e == cudaSuccess) api_count_launch();
  return e;
}

template <int DT, int DP>
cudaError_t dispatch(const AttnParams &p, int32_t *status, cudaStream_t stream) {
  const bool whole = p.c.page_tokens % kTile == 0;
  if (p.group > 8) return whole ? launch<DT, DP, 2, true>(p, status, stream) : launch<DT, DP, 2, false>(p, status, stream);
  return whole ? launch<DT, DP, 1, true>(p, status, stream) : launch<DT, DP, 1, false>(p, status, stream);
}
template <int DT>
cudaError_t dispatch(const AttnParams &p, int32_t *status, cudaStream_t stream) {
  switch (padded_dim(p.c.head_dim)) {
    case 64: return dispatch<DT, 64>(p, status, stream);
    case 128: return dispatch<DT, 128>(p, status, stream);
    default: return dispatch<DT, 256>(p, status, stream);
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
