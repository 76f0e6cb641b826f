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
//     in shared memory (16-byte cp.async, two tiles of 8 KB at 128 elements a head: some 130 KB on
//     their way per SM), with no barrier between warps in the loop.
//   * The unit of work is a tile, not a request: the tiles of all rows and key-value heads form one
//     list, cut evenly over the SMs and over their warps, so the lengths do not have to match anything and one
//     long request fills the GPU as well as many short ones. A warp goes from one (row, head) to the
//     next without draining its ring. Every 32 tiles its lanes work out 32 tiles' places at once.
//   * Consecutive rows of one request (drafted tokens, a prompt) stand beside each other in a tile's columns, as
//     many as the group leaves room for, each with a mask of its own (kShare8 has the rule and the figures).
//   * A (row, head) cut between warps is joined in two steps, in a fixed order: the warps of a CTA, in
//     shared memory, then the CTAs, by the one that finishes last (a counter that it returns to zero).
// What a warp does between two tiles has to stay below the time its share of the bandwidth gives it
// (some 2800 cycles at 8 KB a tile and 8 warps), with room to catch up, so the instructions are few:
//   * Products transposed, S^T = K Q^T and O^T = V^T P^T: tokens (then head elements) are the 16 rows of
//     m16n8k16 and the group's heads its 8 columns, of which a group of 8 fills all. (With the heads
//     as rows, half of every product is padding, and the accumulators twice as many.)
//   * The maximum is not followed exactly: m moves when a score passes it by 2^kSlack, which one vote
//     per tile decides; weights up to 2^kSlack are as exact as those up to 1.
//   * The weights are rounded to the cache's type for the second product. Their remainder, rounded likewise, goes
//     through a second one: 16 significant bits of a weight with bf16, 22 with fp16 (it is off by 2^-16, 2^-22 of itself
//     at most), against the output's 8 and 11. Of 256 requests of up to 4096 tokens one output in 360 is rounded to the
//     other side than the plain form's in fp32 (of which one in 2100 is not the exact value's), and the error against 64
//     bits is the same. A third part would hold fp32's bits: the same time where memory bounds (256 requests), 5 % more
//     for 8 requests of 1000 tokens, 8 % for prompt rows, 12 % for those at 256 elements a head. The sums are the matrix
//     instructions' fp32 accumulators, the exponential is ex2.approx (2 ulp).
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include <algorithm>

#include "serve.cuh"
#include "tc.cuh"

namespace mlora {

namespace {

// Tokens of a tile: 16, and 32 where a head of at most 64 elements makes the tile's copies half as large
// (64 rows of 8 x 64 elements: 41.9 us with 16, 39.8 with 32).
constexpr int tile_tokens(int dp) { return dp == 64 ? 32 : 16; }
constexpr int kRowsPerLaunch = 1024;
// A warp's share of a small call, so that few pieces have to be joined: with 1, 2, 4 tiles, 61 tokens 6.1, 6.4, 7.0 us, 4
// requests of 4 rows 15.5, 15.2, -, 8 rows of 131071 tokens 354, 331, -; the others alike.
constexpr int kMinTiles = 2;
// A CTA's boundary inside a (row, head) of at most kWhole tiles moves to its nearer end, where the CTAs' shares are at
// most kSmallShare tiles, and of at most kWholeLarge where they are larger. Measured (us):
//   kWhole 0, 96, 400: 61 tokens 9.1  6.4  6.5;  300 tokens 11.0  8.8  8.8;  8 requests of 4 rows 20.3  18.7  18.8;  16 requests
//     of 100 to 2000 tokens 19.8  18.6  19.0
//   kWholeLarge 0, 24, 96, 150: 197 short requests of 3 rows 39.7  37.0  34.7  34.8;  64 requests, heads of 64: 41.1  40.2  39.1
//     42.0;  32 requests x 4 rows -  39.4  41.7  41.5;  the same with groups of 8 -  51.1  52.4  52.5;  64 at pages of 1 token
//     -  64.6  66.0  72.5;  32 long requests 81.0  79.8  78.3  79.5
constexpr int kSmallShare = 64, kWhole = 96, kWholeLarge = 24;
constexpr int kMaxGroup = 16;        // query heads of a work item
// Where a warp has at most this many tiles, the list holds an empty one behind every (row, head): what starting
// and ending one costs, about a tile's products (0.5 us), counts beside the tiles then, not in a call that
// waits for memory. Never, at 16, always: 197 requests of 3 rows 45.5  37.0  37.1 us, 37 of 3 rows with a window 24.9  23.0
// 23.0, 256 long requests 210.3  210.0  211.0.
constexpr int kFewTiles = 16;
// Rows of one request share a tile's columns, `group` each, where the SMs have at least kShare8 (row, key-value head)s
// each: up to 8 columns, which costs masks and 1.2 us for the list. From kShare16 on up to 16, twice the products
// and longer joins, if a request's rows need them: their number is the caller's to say (the host sees capacities only:
// 40 requests of 5 rows, groups of 4, in a page table of 256 places 82 us by the capacities, 58 told; 200 decoding rows
// padded to 256, groups of 8, 130 and 125; a prompt of 200 in that table 18.1 and 17.4). Measured (us), 8 heads of 128,
// 500 to 1500 tokens unless said; a row to a tile, 8 columns, 16 columns:
//   group 4: 4 requests x 4 rows (0.8 an SM) 15.3  17.6  22.9;  8 x 4 (1.7) 22.6  18.8  24.2;  64 x 2 (6.7) 71.7  49.9  52.2;
//     32 x 4 (6.7) 55.1  39.7  39.4;  64 x 5 (17) 142  98  83;  16 x 64 (54) 305  189  138;
//     a prompt of 256 (13) 23.1  18.6  19.3, of 1024 (54) 347  232  186
//   group 1: 64 x 8 205  52  54    group 2: 64 x 8 207  75  59    group 8: 32 x 4 (6.7) 55.9  -  51.1
//   group 3, 37 x 3 short ones (3.6) 25.0  23.0  25.6
constexpr int kShare8 = 1, kShare16 = 6;
constexpr float kSlack = 8.f;        // log2 of how far a weight may pass 1 before m moves

constexpr int attn_warps(int dp) { return dp == 256 ? 4 : 8; }
constexpr int attn_stages(int) { return 2; }
// Floats of a partial result: out [16][dp], then m [16] and l [16].
constexpr int partial_floats(int dp) { return kMaxGroup * (dp + 2); }
constexpr int kPartialSlots = 2;  // partial results of a CTA in the workspace
constexpr int padded_dim(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

struct AttnParams {
  mlora_kv_cache c;
  mlora_kv_attn a;
  const uint16_t *k, *v;  // the layer's part of the cache
  FastDiv page;
  int32_t row0, rows;     // this launch's rows
  int32_t group, chunks;  // query heads of a key-value head, in chunks of at most 16
  int32_t pack;           // rows of one request that share a tile's columns, at most
  FastDiv by_group;
  float scale_log2;       // scale * log2(e)
  int32_t *counters;      // [CTAs], zero between calls
  float *partials;        // [CTAs][kPartialSlots][partial_floats]
};

// a / b for a >= 0, b > 0
__device__ __forceinline__ int quick_div(int a, int b) { return (int)((uint32_t)a / (uint32_t)b); }

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

// 0, or NaN where one of the four is an infinity or NaN
__device__ __forceinline__ float odd(const float4 &f) { return (f.x * 0.f + f.y * 0.f) + (f.z * 0.f + f.w * 0.f); }

// acc += x f for a piece's elements f. An infinity or NaN among them, which has come from V, stays what it is when
// the piece's weight x is below the smallest number (where x f is NaN).
__device__ __forceinline__ void add_weighed(float4 &acc, float x, const float4 &f) {
  acc.x += x == 0.f && f.x * 0.f != 0.f ? f.x : x * f.x;
  acc.y += x == 0.f && f.y * 0.f != 0.f ? f.y : x * f.y;
  acc.z += x == 0.f && f.z * 0.f != 0.f ? f.z : x * f.z;
  acc.w += x == 0.f && f.w * 0.f != 0.f ? f.w : x * f.w;
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
__device__ __forceinline__ void cp_async4(void *dst_smem, const void *src_gmem) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst_smem)), "l"(src_gmem) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A tile's place, one per lane for 32 consecutive tiles of the list.
struct Tile {
  // pages of whole 16 tokens: where each 16 of its tokens start in the cache; else [0]: its request and first token
  int64_t off[2];
  uint32_t seen;  // bit t: token t is seen
  uint32_t row;   // the row, with kFirst / kLast for the first / last tile of its (row, head), kNone for no tile
  int32_t hc;     // key-value head and chunk of its group
};
constexpr uint32_t kNone = 1u << 29, kFirst = 1u << 30, kLast = 1u << 31, kRowMask = kNone - 1;

template <int DP, int NW, int NB, bool PACK>
struct AttnSmem {
  static constexpr int kTile = tile_tokens(DP);
  static constexpr int kStages = attn_stages(DP);
  static constexpr int kStageElems = 2 * kTile * DP;  // K, then V
  uint16_t ring[NW][kStages][kStageElems];  // a warp's tiles; after the last, its unfinished last piece
  float head[NW][NB * 8][DP];               // its unfinished first piece
  int32_t first[kRowsPerLaunch + 1];        // tiles (of one head) before a row
  int32_t pos[kRowsPerLaunch];              // last token seen; -1: none, -2: a bad row
  // PACK, of a pack's first row: the first and the last token that its rows see, and their number (0: not a first row)
  int32_t low[PACK ? kRowsPerLaunch : 1], high[PACK ? kRowsPerLaunch : 1];
  uint8_t rows[PACK ? kRowsPerLaunch : 1];
  int32_t req[kRowsPerLaunch];              // the row's request
  uint32_t seen[NW][kStages];               // bit t: token t of the tile is seen
  int32_t warp_sum[NW], warp_rows[NW];
  int32_t page_id[NW][2 * kStages][kTile];  // pages of tokens, where a page does not hold whole tiles
  int64_t at[NW][kTile];                    // and the tokens' places in the cache (-1: not seen)
  // pieces: [2w] without the first tile of its (row, head), [2w+1] with it
  float m[2 * NW][kMaxGroup], l[2 * NW][kMaxGroup];
  int32_t piece_row[2 * NW], piece_hc[2 * NW];
  int32_t last[2];
};

// The last row with first[row] HC <= x, for x below the list's length.
__device__ __forceinline__ int row_of(const int32_t *first, int rows, int HC, int x) {
  int r = 0;
  for (int hi = rows; hi - r > 1;) {
    const int mid = (r + hi) >> 1;
    if (first[mid] * HC <= x) r = mid;
    else hi = mid;
  }
  return r;
}

// Columns of the item (row r, head and chunk hc), and the first's query head. rows: a pack's, by its first row.
template <bool PACK>
__device__ __forceinline__ int columns(const AttnParams &p, const uint8_t *rows, int r, int hc, int64_t &head0) {
  const int hk = p.chunks == 1 ? hc : hc / p.chunks, g0 = p.chunks == 1 ? 0 : (hc - hk * p.chunks) * kMaxGroup;
  head0 = (int64_t)hk * p.group + g0;
  if (PACK) return rows[r] * p.group;  // (one chunk)
  return min(p.group - g0, kMaxGroup);
}

template <int DT>
__device__ __forceinline__ bool is_wild(uint32_t x) {  // the 16-bit number in its low half is an infinity or NaN
  constexpr uint32_t kExp = DT == MLORA_FP16 ? 0x7C00u : 0x7F80u;
  return (x & kExp) == kExp;
}

// An infinity or NaN in a token's V. The products leave NaN for an infinity as soon as a part of its weight is 0 (what
// remains of an exact weight) or negative (a remainder), or o is rescaled by 0. So where a piece's o is not finite, the V
// of the warp's pieces are read again, and an element that holds infinities or NaN becomes their sum over the tokens that
// the column sees: whatever a weight above 0 is, an infinity with it is that infinity. The others stay as they are. Twice
// over the tokens, to clear such elements where they have been left and to sum them there. Tiles w0 .. w0 + n - 1 of the
// list are the warp's. (A function of its own: inside the kernel its registers were the loop's, and 4 requests of 512
// rows took 457 us instead of 434.)
template <int DT, int DP, int NB, bool PACK>
__device__ __noinline__ void mend_values(const AttnParams &p, AttnSmem<DP, attn_warps(DP), NB, PACK> &sh, int w0, int n,
                                         int empty) {
  constexpr int kTile = AttnSmem<DP, attn_warps(DP), NB, PACK>::kTile;
  const mlora_kv_attn &a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = p.c.head_dim, HC = p.c.num_kv_heads * p.chunks;
  auto low_of = [&](int pos) { return a.window ? max(0, pos + 1 - a.window) : 0; };
  auto wild2 = [&](uint32_t x) { return is_wild<DT>(x) || is_wild<DT>(x >> 16); };
  __syncwarp();
#pragma unroll 1
  for (int x = w0; x < w0 + n;) {
    const int r = row_of(sh.first, p.rows, HC, x), nt = sh.first[r + 1] - sh.first[r], rem = x - sh.first[r] * HC;
    const int item = quick_div(rem, nt), tile0 = rem - item * nt, tiles = min(nt - empty - tile0, w0 + n - x);
    x += nt - tile0;
    if (tiles <= 0) continue;
    const bool whole = tile0 == 0 && tiles == nt - empty;
    float *const part = tile0 == 0 ? reinterpret_cast<float *>(sh.ring[warp]) : sh.head[warp][0];
    const int high = PACK ? sh.high[r] : sh.pos[r], low = PACK ? sh.low[r] : low_of(high);
    const int from = max(low, (low / kTile + tile0) * kTile), last = (low / kTile + tile0 + tiles - 1) * kTile;
    const int tokens = last - from + min(high - last, kTile - 1) + 1;
    int64_t head0;
    const int cols = columns<PACK>(p, sh.rows, r, item, head0);
    const int32_t *const pages = a.page_table + (int64_t)sh.req[r] * a.table_stride;
    const uint16_t *const v = p.v + (int64_t)(p.chunks == 1 ? item : item / p.chunks) * p.c.head_stride;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass)
#pragma unroll 1
      for (int i0 = 0; i0 < tokens; i0 += 32) {
        // a lane's token: whether its V holds any
        const uint16_t *mine = v;
        bool some = false;
        if (i0 + lane < tokens) {
          const int t = from + i0 + lane, pg = div_by(p.page, t), id = pages[pg];
          if (id >= 0 && id < p.c.num_pages) {
            mine += (int64_t)id * p.c.page_stride + (int64_t)(t - pg * p.page.d) * p.c.token_stride;
#pragma unroll 4
            for (int i = 0; i < D / 8; ++i) {
              const uint4 y = ldg_u4(mine + i * 8);
              some |= wild2(y.x) || wild2(y.y) || wild2(y.z) || wild2(y.w);
            }
          }
        }
#pragma unroll 1
        for (uint32_t left = __ballot_sync(~0u, some); left; left &= left - 1) {
          const int k = __ffs(left) - 1, t = from + i0 + k;
          const uint16_t *const of =
              reinterpret_cast<const uint16_t *>(__shfl_sync(~0u, reinterpret_cast<unsigned long long>(mine), k));
#pragma unroll 1
          for (int d = lane; d < D; d += 32) {  // (a lane comes back to the elements that it has cleared)
            const uint32_t y = of[d];
            if (!is_wild<DT>(y)) continue;
#pragma unroll 1
            for (int c = 0; c < cols; ++c) {
              const int row = r + (PACK ? div_by(p.by_group, c) : 0);
              if (PACK && (t > sh.pos[row] || t < low_of(sh.pos[row]))) continue;
              if (whole) {
                uint16_t *const to = static_cast<uint16_t *>(a.out) + ((int64_t)p.row0 + row) * a.ldo +
                                     (head0 + c - (row - r) * p.group) * D + d;
                *to = pass ? Elem<DT>::from_float(Elem<DT>::lo(*to) + Elem<DT>::lo(y)) : (uint16_t)0;
              } else {
                float &to = part[c * DP + d];
                to = pass ? to + Elem<DT>::lo(y) : 0.f;
              }
            }
          }
        }
      }
  }
}

// PAGED16: a page holds whole tiles. NB: blocks of 8 columns (heads of a group's chunk). PACK: rows of one request share
// them.
template <int DT, int DP, int NB, bool PAGED16, bool PACK>
__global__ void __launch_bounds__(attn_warps(DP) * 32, 1)
    kv_attention_kernel(const __grid_constant__ AttnParams p, int32_t *status) {
  constexpr int NW = attn_warps(DP), NT = NW * 32;
  using Smem = AttnSmem<DP, NW, NB, PACK>;
  constexpr int S = Smem::kStages, kTile = Smem::kTile, H = kTile / 16;  // H halves of 16 tokens
  constexpr uint32_t kAll = kTile == 32 ? ~0u : 0xFFFFu;
  constexpr int CH = DP / 8;    // 16-byte chunks of a token's head
  constexpr int GP = NB * 8;    // heads that a piece holds
  static_assert(GP * DP * 4 <= S * Smem::kStageElems * 2, "a piece fits in the ring");
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
  int empty;  // 1: an empty tile behind every (row, head)
  auto low_of = [&](int pos) { return a.window ? max(0, pos + 1 - a.window) : 0; };  // the first token that is seen
  {
    const int each = (R + NT - 1) / NT, r0 = min(tid * each, R), r1 = min(r0 + each, R);
    int sum = 0, some = 0, bad = 0;  // tiles; rows that have any
    for (int r = r0; r < r1; ++r) {
      const int64_t row = (int64_t)p.row0 + r;
      int pos = a.position[row], n = 0;
      const int req = a.row_request ? a.row_request[row] : (int)row;
      if (pos < -1 || pos >= (int64_t)a.max_pages * p.page.d) bad |= MLORA_STATUS_BAD_LENGTH, pos = -2;
      else if (pos >= 0 && (req < 0 || req >= a.num_requests)) bad |= MLORA_STATUS_BAD_REQUEST, pos = -2;
      sh.pos[r] = pos;
      sh.req[r] = req;
      if (PACK) continue;
      if (pos >= 0) n = pos / kTile - low_of(pos) / kTile + 1;
      sh.first[r] = n;
      sum += n;
      some += n > 0;
    }
    if (PACK) {
      // Rows that follow each other, of one request, whose tokens overlap or touch, are a run; its rows from the
      // first, p.pack at a time, are packs. A pack's first row stands for it; the others have no tiles.
      auto starts_run = [&](int r) {
        return r == 0 || sh.pos[r] < 0 || sh.pos[r - 1] < 0 || sh.req[r] != sh.req[r - 1] ||
               low_of(sh.pos[r]) > sh.pos[r - 1] + 1 || sh.pos[r] + 1 < low_of(sh.pos[r - 1]);
      };
      __syncthreads();
      int last = -1;
      for (int r = r0; r < r1; ++r)
        if (starts_run(r)) last = r;
      int upto = last;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(~0u, upto, d);
        if (lane >= d) upto = max(upto, x);
      }
      if (lane == 31) sh.warp_sum[warp] = upto;
      int run = __shfl_up_sync(~0u, upto, 1);
      if (lane == 0) run = -1;
      __syncthreads();
      for (int w = 0; w < warp; ++w) run = max(run, sh.warp_sum[w]);
      for (int r = r0; r < r1; ++r) {
        if (starts_run(r)) run = r;
        int lo = low_of(sh.pos[r]), hi = sh.pos[r], count = 0, n = 0;
        if ((r - run) % p.pack == 0) {
          for (count = 1; count < p.pack && r + count < R && !starts_run(r + count); ++count) {
            lo = min(lo, low_of(sh.pos[r + count]));
            hi = max(hi, sh.pos[r + count]);
          }
          n = hi >= 0 ? hi / kTile - lo / kTile + 1 : 0;
        }
        sh.low[r] = lo, sh.high[r] = hi, sh.rows[r] = count, sh.first[r] = n;
        sum += n;
        some += n > 0;
      }
      __syncthreads();
    }
    int incl = sum, rows = some;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(~0u, incl, d), y = __shfl_up_sync(~0u, rows, d);
      if (lane >= d) incl += x, rows += y;
    }
    if (lane == 31) sh.warp_sum[warp] = incl, sh.warp_rows[warp] = rows;
    if (bad && blockIdx.x == 0) report(status, bad);
    if (tid < 2 * NW) sh.piece_row[tid] = -1;
    __syncthreads();
    int at = incl - sum, before = rows - some, all = 0;
    for (int w = 0; w < NW; ++w) {
      if (w < warp) at += sh.warp_sum[w], before += sh.warp_rows[w];
      all += sh.warp_sum[w];
    }
    empty = (int64_t)all * HC <= (int64_t)gridDim.x * NW * kFewTiles ? 1 : 0;
    at += empty * before;
    for (int r = r0; r < r1; ++r) {
      const int n = sh.first[r];
      sh.first[r] = at;
      at += n ? n + empty : 0;
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
  // Even shares: the first `rest` CTAs (warps) take a tile more.
  const int T = sh.first[R] * HC;  // (below 2^31: the launcher sees to it)
  const int C = min((int)gridDim.x, quick_div(T + kMinTiles - 1, kMinTiles));
  if ((int)blockIdx.x >= C) return;
  const int share = quick_div(T, C), rest = T - share * C;
  auto first_of = [&](int cta) { return cta * share + min(cta, rest); };
  auto cta_of = [&](int tile) {
    const int longer = rest * (share + 1);
    return tile < longer ? quick_div(tile, share + 1) : rest + quick_div(tile - longer, share);
  };
  auto row_of = [&](int x) { return mlora::row_of(sh.first, R, HC, x); };
  int t0, t1;
  {
    int x = first_of(blockIdx.x + (lane & 1));  // lanes 0 and 1: the CTA's two boundaries
    if (x < T) {
      const int r = row_of(x), nt = sh.first[r + 1] - sh.first[r];
      if (nt <= (share <= kSmallShare ? kWhole : kWholeLarge)) {
        const int rem = x - sh.first[r] * HC, in = rem - quick_div(rem, nt) * nt;
        x += 2 * in < nt ? -in : nt - in;
      }
    }
    t0 = __shfl_sync(~0u, x, 0), t1 = __shfl_sync(~0u, x, 1);
  }
  const int mine = t1 - t0;
  const int nw = min(NW, max(1, quick_div(mine + kMinTiles - 1, kMinTiles)));
  const int each = quick_div(mine, nw), over = mine - each * nw;
  const int w0 = t0 + warp * each + min(warp, over);
  const int n = warp < nw ? each + (warp < over ? 1 : 0) : 0;

  // The columns of an item (row r, head and chunk hc): the query heads of its chunk, or those of its pack's rows. Head
  // head0 of row r is the first; column c is head in(c) behind it, of row below(c) behind r.
  auto columns = [&](int r, int hc, int64_t &head0) { return mlora::columns<PACK>(p, sh.rows, r, hc, head0); };
  auto below = [&](int c) { return PACK ? div_by(p.by_group, c) : 0; };
  auto in = [&](int c) { return c - below(c) * p.group; };
  auto lse_of = [&](float m, float l) { return l == 0.f ? -CUDART_INF_F : (m - kShift) * CUDART_LN2_F + logf(l); };
  float *const partials = p.partials + (int64_t)blockIdx.x * kPartialSlots * partial_floats(DP);
  // chunks past the head's end are never copied: zero for good
  if (D < DP) {
    for (int i = lane; i < S * Smem::kStageElems / 8; i += 32)
      reinterpret_cast<uint4 *>(sh.ring[warp])[i] = make_uint4(0, 0, 0, 0);
    __syncwarp();
  }
  int pieces = 0;
  if (n > 0) {
    // tiles w0 + 32 b + lane
    auto place = [&](int b) {
      Tile t{};
      const int i = b * 32 + lane, x = w0 + i;
      if (i >= n) return t;
      const int r = row_of(x);
      const int nt = sh.first[r + 1] - sh.first[r];
      const int rem = x - sh.first[r] * HC;
      t.hc = rem < nt ? 0 : quick_div(rem, nt);
      const int tile = rem - t.hc * nt;
      if (empty && tile == nt - 1) {
        t.row = kNone;
        return t;
      }
      const int pos = PACK ? sh.high[r] : sh.pos[r], lo = PACK ? sh.low[r] : low_of(pos);
      const int t0 = (lo / kTile + tile) * kTile;
      t.seen = kAll;
      if (t0 < lo) t.seen &= kAll << (lo - t0);
      if (pos - t0 < kTile - 1) t.seen &= (2u << (pos - t0)) - 1u;
      t.row = (uint32_t)r | (tile == 0 ? kFirst : 0u) | (tile == nt - 1 - empty ? kLast : 0u);
      const int64_t row = (int64_t)p.row0 + r;
      const int req = sh.req[r];
      if (tile == 0 || i == 0) {  // q of the (row, head), into L2
        int64_t head0;
        const int heads = min(columns(r, t.hc, head0), p.group);
        for (int k = 0; k < (PACK ? sh.rows[r] : 1); ++k)
          prefetch_l2(static_cast<const uint16_t *>(a.q) + (row + k) * a.ldq + head0 * D, (uint32_t)(heads * D * 2));
      }
      if constexpr (PAGED16) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
          if (!((t.seen >> (16 * h)) & 0xFFFFu)) continue;
          const int pg = div_by(p.page, t0 + 16 * h);
          const int id = a.page_table[(int64_t)req * a.table_stride + pg];
          if (id >= 0 && id < p.c.num_pages) {
            t.off[h] = (int64_t)id * p.c.page_stride + (int64_t)(t0 + 16 * h - pg * p.page.d) * p.c.token_stride +
                       (int64_t)(p.chunks == 1 ? t.hc : t.hc / p.chunks) * p.c.head_stride;
          } else {
            report(status, MLORA_STATUS_BAD_PAGE);
            t.seen &= ~(0xFFFFu << (16 * h));
          }
        }
      } else {
        t.off[0] = ((int64_t)req << 32) | (uint32_t)t0;
      }
      return t;
    };
    Tile cur = place(0), nxt{};
    if (n > 32) nxt = place(1);
    int cur_batch = 0;
    auto tile_at = [&](int i) -> const Tile & { return (i >> 5) == cur_batch ? cur : nxt; };

    // ---- loads, S - 1 tiles ahead of the products --------------------------------------------------
    const int lt = lane / CH, lc = lane % CH;  // a lane's token and chunk within a step of 32 chunks
    constexpr int kStep = 32 / CH;             // tokens of such a step
    const bool copies = lc * 8 < D;
    // Pages of other sizes: the page of each token of a tile, copied to shared memory S tiles before
    // the tile's own copies start (with the copies of a tile that is waited for before that).
    auto look_up = [&](int i) {
      const Tile &b = tile_at(i);
      const int64_t at = __shfl_sync(~0u, b.off[0], i & 31);
      const uint32_t range = __shfl_sync(~0u, b.seen, i & 31);
      const int t = (int)(uint32_t)at + lane;
      if (lane < kTile && ((range >> lane) & 1u))
        cp_async4(&sh.page_id[warp][i % (2 * S)][lane], a.page_table + (at >> 32) * a.table_stride + div_by(p.page, t));
    };
    auto issue = [&](int i, int slot) {  // tile i into ring slot `slot`
      uint16_t *ks = sh.ring[warp][slot];
      if constexpr (PAGED16) {
        const Tile &b = tile_at(i);
        const uint32_t seen = __shfl_sync(~0u, b.seen, i & 31);
        if (lane == 0) sh.seen[warp][slot] = seen;
        const bool none = (__shfl_sync(~0u, b.row, i & 31) & kNone) != 0;
#pragma unroll
        for (int h = 0; h < H; ++h) {
          const int64_t off = __shfl_sync(~0u, b.off[h], i & 31);
          if (!copies || none) continue;  // (a tile whose page is missing is filled with zeros)
          const int64_t at = off + (int64_t)lt * p.c.token_stride + lc * 8;
          const uint16_t *pk = p.k + at, *pv = p.v + at;
          const int64_t step = kStep * p.c.token_stride;
#pragma unroll
          for (int j = 0; j < 16 / kStep; ++j) {
            const int t = 16 * h + j * kStep + lt;
            uint16_t *dst = ks + t * DP + ((lc ^ (t & 7)) * 8);
            const uint32_t bytes = (seen >> t) & 1u ? 16u : 0u;
            tc::cp_async16(dst, bytes ? pk : p.k, bytes);
            tc::cp_async16(dst + kTile * DP, bytes ? pv : p.v, bytes);
            pk += step, pv += step;
          }
        }
      } else {
        const Tile &b = tile_at(i);
        const int hc = __shfl_sync(~0u, b.hc, i & 31);
        const int t0 = (int)(uint32_t)__shfl_sync(~0u, b.off[0], i & 31) + lane % kTile;
        const bool want = (__shfl_sync(~0u, b.seen, i & 31) >> (lane % kTile)) & 1u;
        const int id = want ? sh.page_id[warp][i % (2 * S)][lane % kTile] : -1;
        const bool good = id >= 0 && id < p.c.num_pages;
        if (want && !good) report(status, MLORA_STATUS_BAD_PAGE);
        if (lane < kTile)
          sh.at[warp][lane] = good ? (int64_t)id * p.c.page_stride +
                                         (int64_t)(t0 - div_by(p.page, t0) * p.page.d) * p.c.token_stride +
                                         (int64_t)(p.chunks == 1 ? hc : hc / p.chunks) * p.c.head_stride
                                   : -1;
        const uint32_t seen = __ballot_sync(~0u, good) & kAll;  // (also orders at[] for the warp)
        __syncwarp();
        if (lane == 0) sh.seen[warp][slot] = seen;
        if (copies) {
#pragma unroll
          for (int j = 0; j < kTile / kStep; ++j) {
            const int t = j * kStep + lt;
            const int64_t o = sh.at[warp][t];
            const uint32_t bytes = o >= 0 ? 16u : 0u;
            const int64_t from = o >= 0 ? o + lc * 8 : 0;
            uint16_t *dst = ks + t * DP + ((lc ^ (t & 7)) * 8);
            tc::cp_async16(dst, p.k + from, bytes);
            tc::cp_async16(dst + kTile * DP, p.v + from, bytes);
          }
        }
        __syncwarp();  // at[] may be written again
        if (i + S < n) look_up(i + S);
      }
    };
    if constexpr (!PAGED16) {
      for (int i = 0; i < min(S, n); ++i) look_up(i);
      cp_async_commit();
      cp_async_wait<0>();
      __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
      if (i < n) issue(i, i);
      cp_async_commit();
    }

    // ---- products ----------------------------------------------------------------------------------
    const int g = lane >> 2, quad = lane & 3;
    uint32_t q[DP / 16][NB][2];  // Q^T: head elements kk * 16 + {0, 8} + quad * 2 + {0, 1}, head g of the block
    uint32_t ahead[DP / 16][NB][2];  // the next (row, head)'s, on its way while the last tile before it is computed
    auto load_q = [&](int i) {
      const Tile &b = tile_at(i);
      const int r = (int)(__shfl_sync(~0u, b.row, i & 31) & kRowMask);
      int64_t h0;
      const int cols = columns(r, __shfl_sync(~0u, b.hc, i & 31), h0);
      const uint16_t *qr[NB];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int c = min(nb * 8 + g, cols - 1);
        qr[nb] = static_cast<const uint16_t *>(a.q) + ((int64_t)p.row0 + r + below(c)) * a.ldq + (h0 + in(c)) * D;
      }
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int d = kk * 16 + j * 8 + quad * 2;
            ahead[kk][nb][j] = nb * 8 + g < cols && d < D ? *reinterpret_cast<const uint32_t *>(qr[nb] + d) : 0u;
          }
    };
    bool mend = false;  // a piece's o holds an infinity or NaN
    constexpr bool kAhead = DP * NB < 512;  // (no registers left for it at 16 heads of 256)
    float o[DP / 16][NB][4];     // O^T: elements j * 16 + g (0, 1) and + 8 (2, 3), heads quad * 2 + {0, 1}
    float m[NB][2], l[NB][2];    // of heads quad * 2 + {0, 1}; l: of this lane's tokens
    bool start = true, with_first = false;
    int token = 0, sees[NB][2];  // packed rows: the tile's token g, and the last token that a column sees
    int row_in = 0, hc = 0, gn = 0;
    int64_t row = 0, head0 = 0;
    // lane's row and chunk in ldmatrix: K (token, plain) and V (token, transposed)
    const int kt = lane & 15, kc = lane >> 4;
    const int vt = (lane & 7) + ((lane >> 4) << 3), vc = (lane >> 3) & 1;
    int slot = 0;
    {
      const int skip = __shfl_sync(~0u, cur.row, 0) & kNone ? 1 : 0;
      if (kAhead && skip < n) load_q(skip);
    }
    for (int it = 0; it < n; ++it) {
      if ((it & 31) == 0 && it) {
        cur = nxt;
        ++cur_batch;
        if (it + 32 < n) nxt = place(cur_batch + 1);
      }
      const uint32_t meta = __shfl_sync(~0u, cur.row, it & 31);
      if (start && !(meta & kNone)) {
        if constexpr (!kAhead) load_q(it);
        row_in = (int)(meta & kRowMask);
        hc = __shfl_sync(~0u, cur.hc, it & 31);
        with_first = (meta & kFirst) != 0;
        row = (int64_t)p.row0 + row_in;
        gn = columns(row_in, hc, head0);
        if (PACK) {
          const int nt = sh.first[row_in + 1] - sh.first[row_in];
          token = (sh.low[row_in] / kTile + (w0 + it - sh.first[row_in] * HC - hc * nt)) * kTile + g;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int j = 0; j < 2; ++j) sees[nb][j] = sh.pos[row_in + below(min(nb * 8 + quad * 2 + j, gn - 1))];
        }
#pragma unroll
        for (int kk = 0; kk < DP / 16; ++kk)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) q[kk][nb][0] = ahead[kk][nb][0], q[kk][nb][1] = ahead[kk][nb][1];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
          for (int j = 0; j < DP / 16; ++j) o[j][nb][0] = o[j][nb][1] = o[j][nb][2] = o[j][nb][3] = 0.f;
          m[nb][0] = m[nb][1] = -CUDART_INF_F;
          l[nb][0] = l[nb][1] = 0.f;
        }
        start = false;
      }
      if (kAhead && (meta & kLast) && it + 1 + empty < n) load_q(it + 1 + empty);  // another (row, head)'s
      if (it + S - 1 < n) issue(it + S - 1, slot == 0 ? S - 1 : slot - 1);
      cp_async_commit();
      cp_async_wait<S - 1>();
      __syncwarp();
      if (meta & kNone) {
        if (++slot == S) slot = 0;
        __syncwarp();
        continue;
      }
      const uint32_t seen = sh.seen[warp][slot];
      const uint32_t ks = smem_u32(sh.ring[warp][slot]), vs = ks + kTile * DP * 2;

      float s[H][NB][4] = {}, s2[H][NB][4] = {};  // two chains of products
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk)
#pragma unroll
        for (int h = 0; h < H; ++h) {
          uint32_t x[4];
          ldmatrix4(x, ks + (16 * h + kt) * DP * 2 + (((kk * 2 + kc) ^ (kt & 7)) << 4));
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) mma<DT>(kk & 1 ? s2[h][nb] : s[h][nb], x, q[kk][nb][0], q[kk][nb][1]);
        }
      // s[h][nb][2 i + j]: token 16 h + g + 8 i, head quad * 2 + j
      bool past = false, part = false;  // part: a token that only some columns see
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            bool on = ((seen >> (16 * h + g + 8 * (j >> 1))) & 1u) != 0;
            if (PACK) {
              const int t = token + 16 * h + 8 * (j >> 1), last = sees[nb][j & 1];
              const bool sees_it = t <= last && t >= low_of(last);
              part |= on && !sees_it;
              on = on && sees_it;
            }
            s[h][nb][j] = on ? (s[h][nb][j] + s2[h][nb][j]) * p.scale_log2 : -CUDART_INF_F;
            past |= s[h][nb][j] > m[nb][j & 1] + kSlack;
          }
      if (PACK && __any_sync(~0u, part)) {
        // A column that does not see a token has its weight 0, and 0 times an infinity or NaN of its V is NaN. Those
        // elements leave the tile and mark the columns that do see them (mend_values goes by that).
        uint16_t *const v = sh.ring[warp][slot] + kTile * DP;
        bool some = false;
        for (int i = lane; i < kTile * DP / 2; i += 32) {
          const uint32_t x = reinterpret_cast<const uint32_t *>(v)[i];
          some |= is_wild<DT>(x) || is_wild<DT>(x >> 16);
        }
        if (__any_sync(~0u, some)) {
#pragma unroll 1
          for (int t = 0; t < kTile; ++t) {
            const int at = token - g + t;
#pragma unroll
            for (int j = 0; j < DP / 8; ++j) {
              const uint32_t x = v[t * DP + ((j ^ (t & 7)) << 3) + g];  // element 8 j + g
              if (!is_wild<DT>(x)) continue;
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                  if (((seen >> t) & 1u) && at <= sees[nb][i] && at >= low_of(sees[nb][i]))
                    o[j / 2][nb][(j & 1) * 2 + i] += Elem<DT>::lo(x);
            }
          }
          __syncwarp();
          for (int i = lane; i < kTile * DP; i += 32)
            if (is_wild<DT>(v[i])) v[i] = 0;
          __syncwarp();
        }
      }
      token += kTile;
      if (__any_sync(~0u, past)) {  // m moves to the maximum
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float top = fmaxf(s[0][nb][j], s[0][nb][j + 2]);
            if (H > 1) top = fmaxf(top, fmaxf(s[H - 1][nb][j], s[H - 1][nb][j + 2]));
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
      uint32_t hi[H][NB][2], lo[H][NB][2];  // P^T: tokens 16 h + {0, 8} + quad * 2 + {0, 1}, head g
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float base = m[nb][j & 1] == -CUDART_INF_F ? 0.f : m[nb][j & 1] - kShift;
            w[j] = exp2_fast(s[h][nb][j] - base);
            l[nb][j & 1] += w[j];
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t big, left;
            split_pair<DT>(w[2 * i], w[2 * i + 1], big, left);
            hi[h][nb][i] = transpose8(big);
            lo[h][nb][i] = transpose8(left);
          }
        }
#pragma unroll
      for (int j = 0; j < DP / 16; ++j)
#pragma unroll
        for (int h = 0; h < H; ++h) {
          uint32_t x[4];
          ldmatrix4_t(x, vs + (16 * h + vt) * DP * 2 + (((j * 2 + vc) ^ (vt & 7)) << 4));
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            mma<DT>(o[j][nb], x, hi[h][nb][0], hi[h][nb][1]);
            mma<DT>(o[j][nb], x, lo[h][nb][0], lo[h][nb][1]);
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
        {
          float not_finite[4] = {};  // 0, or NaN where o holds an infinity or NaN
#pragma unroll
          for (int i = 0; i < DP / 16; ++i)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int j = 0; j < 4; ++j) not_finite[j] = fmaf(o[i][nb][j], 0.f, not_finite[j]);
          mend |= __any_sync(~0u, (not_finite[0] + not_finite[1]) + (not_finite[2] + not_finite[3]) != 0.f) != 0;
        }
        if ((meta & kLast) && with_first) {  // and whole
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            float inv[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              inv[j] = l[nb][j] == 0.f ? 0.f : 1.f / l[nb][j];
              const int c = nb * 8 + quad * 2 + j;
              if (a.lse && g == 0 && c < gn)
                a.lse[(row + below(c)) * a.num_q_heads + head0 + in(c)] = lse_of(m[nb][j], l[nb][j]);
            }
            // from head elements as rows to heads as rows: elements j * 8 + quad * 2 + {0, 1} of head g
            const int c = min(nb * 8 + g, gn - 1);
            uint16_t *dst = static_cast<uint16_t *>(a.out) + (row + below(c)) * a.ldo + (head0 + in(c)) * D + quad * 2;
#pragma unroll
            for (int j = 0; j < DP / 8; ++j) {
              const float *x = &o[j / 2][nb][(j & 1) * 2];
              const uint32_t two = transpose8((uint32_t)Elem<DT>::from_float(x[0] * inv[0]) |
                                              ((uint32_t)Elem<DT>::from_float(x[1] * inv[1]) << 16));
              if (j * 8 < D && nb * 8 + g < gn) *reinterpret_cast<uint32_t *>(dst + j * 8) = two;
            }
          }
        } else {
          // with the first tile it is the warp's last piece, and the ring is idle
          const int piece = 2 * warp + (with_first ? 1 : 0);
          float *part = with_first ? reinterpret_cast<float *>(sh.ring[warp]) : sh.head[warp][0];
          if (with_first) {
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
          if (lane == 0) sh.piece_row[piece] = row_in, sh.piece_hc[piece] = hc;
          pieces = 1;
        }
      }
    }
    cp_async_wait<0>();
    if (mend) mend_values<DT, DP, NB, PACK>(p, sh, w0, n, empty);
  }
  if (!__syncthreads_or(pieces)) return;

  // ---- join the pieces of the CTA's warps, then those of the CTAs ------------------------------------
  // Every warp finds the runs of pieces of one (row, head) (lane e looks at piece e) and joins some of their
  // heads. A run that began in an earlier CTA, and one that goes on in a later one, become the CTA's
  // partial results 0 and 1; the others are done.
  const int my_row = lane < 2 * nw ? sh.piece_row[lane] : -1, my_hc = lane < 2 * nw ? sh.piece_hc[lane] : 0;
  const uint32_t any = __ballot_sync(~0u, my_row >= 0);
  uint32_t starts;
  {
    const uint32_t below = any & ((1u << lane) - 1u);
    const int before = below ? 31 - __clz(below) : 0;
    const int r0 = __shfl_sync(~0u, my_row, before), c_before = __shfl_sync(~0u, my_hc, before);
    starts = __ballot_sync(~0u, my_row >= 0 && (!below || r0 != my_row || c_before != my_hc));
  }
  auto pack4 = [&](float4 f) {
    uint2 u;
    u.x = (uint32_t)Elem<DT>::from_float(f.x) | ((uint32_t)Elem<DT>::from_float(f.y) << 16);
    u.y = (uint32_t)Elem<DT>::from_float(f.z) | ((uint32_t)Elem<DT>::from_float(f.w) << 16);
    return u;
  };
  auto warp_max = [&](float x) {
#pragma unroll
    for (int d = 16; d; d >>= 1) x = fmaxf(x, __shfl_xor_sync(~0u, x, d));
    return x;
  };
  auto warp_sum = [&](float x) {
#pragma unroll
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(~0u, x, d);
    return x;
  };
  // of the run that this lane's piece belongs to
  const bool valid = my_row >= 0;
  const int lead = valid ? 31 - __clz(starts & ((2u << lane) - 1u)) : 0;
  const uint32_t later = lane == 31 ? 0u : starts >> (lane + 1);
  const uint32_t run = valid ? any & (~0u << lead) & (later ? (2u << (lane + __ffs(later) - 1)) - 1u : ~0u) : 0u;
  bool here = false, done = false;
  int heads = 0;
  int64_t head0 = 0;
  if (valid) {
    const int nt = sh.first[my_row + 1] - sh.first[my_row], begin = sh.first[my_row] * HC + my_hc * nt;
    here = begin >= t0, done = here && begin + nt - empty <= t1;
    heads = columns(my_row, my_hc, head0);
  }
  const int64_t my_out = done ? ((int64_t)p.row0 + my_row) * a.ldo + head0 * D : here * (int64_t)partial_floats(DP);
  for (int head = warp; head < GP; head += NW) {  // (a column)
    float top = -CUDART_INF_F, sum = 0.f, w = 0.f;
    if (head < heads) {
      for (uint32_t left = run; left; left &= left - 1) top = fmaxf(top, sh.m[__ffs(left) - 1][head]);
      const float base = top == -CUDART_INF_F ? 0.f : top;
      for (uint32_t left = run; left; left &= left - 1) {
        const int e = __ffs(left) - 1;
        sum += exp2_fast(sh.m[e][head] - base) * sh.l[e][head];
      }
      w = exp2_fast(sh.m[lane][head] - base);
      if (done) w *= sum == 0.f ? 0.f : 1.f / sum;
      if (lane == lead) {
        if (!done) {
          float *to = partials + my_out + kMaxGroup * DP + head;
          to[0] = top, to[16] = sum;
        } else if (a.lse) {
          a.lse[((int64_t)p.row0 + my_row + below(head)) * a.num_q_heads + head0 + in(head)] = lse_of(top, sum);
        }
      }
    }
    for (uint32_t todo = starts; todo; todo &= todo - 1) {
      const int at = __ffs(todo) - 1;
      const uint32_t pieces_of = __shfl_sync(~0u, run, at);
      const int flags = __shfl_sync(~0u, heads * 2 + (done ? 1 : 0), at);
      const int64_t out = __shfl_sync(~0u, my_out, at);
      if (head >= flags >> 1) continue;
#pragma unroll
      for (int i0 = 0; i0 < DP / 4; i0 += 32) {
        const int i = i0 + lane;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        auto piece = [&](int e) {
          return reinterpret_cast<const float4 *>(e & 1 ? reinterpret_cast<const float *>(sh.ring[e >> 1])
                                                        : sh.head[e >> 1][0])[head * (DP / 4) + i];
        };
        for (uint32_t left = pieces_of; left; left &= left - 1) {
          const int e = __ffs(left) - 1;
          const float x = __shfl_sync(~0u, w, e);
          if (i < DP / 4) {
            const float4 f = piece(e);
            acc.x += x * f.x, acc.y += x * f.y, acc.z += x * f.z, acc.w += x * f.w;
          }
        }
        if (__any_sync(~0u, odd(acc) != 0.f)) {
          acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
          for (uint32_t left = pieces_of; left; left &= left - 1) {
            const int e = __ffs(left) - 1;
            const float x = __shfl_sync(~0u, w, e);
            if (i < DP / 4) add_weighed(acc, x, piece(e));
          }
        }
        if (i >= DP / 4) continue;
        if (!(flags & 1)) reinterpret_cast<float4 *>(partials + out)[head * (DP / 4) + i] = acc;
        else if (i * 4 < D)
          *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + out + below(head) * a.ldo + in(head) * D + i * 4) =
              pack4(acc);
      }
    }
  }
  int open_row[2] = {-1, -1}, open_hc[2];
  {
    const int one = __ffs(starts) - 1, end = 31 - __clz(starts);  // the first and the last run
    const int flags = (here ? 1 : 0) | (done ? 2 : 0);
    if (!(__shfl_sync(~0u, flags, one) & 1)) open_row[0] = __shfl_sync(~0u, my_row, one);
    open_hc[0] = __shfl_sync(~0u, my_hc, one);
    if (__shfl_sync(~0u, flags, end) == 1) open_row[1] = __shfl_sync(~0u, my_row, end);
    open_hc[1] = __shfl_sync(~0u, my_hc, end);
  }
  if (open_row[0] < 0 && open_row[1] < 0) return;
  __syncthreads();
  int c0[2], c1[2];  // first and last CTA of the items this CTA shares with others
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (open_row[h] < 0) continue;
    const int r = open_row[h];
    const int nt = sh.first[r + 1] - sh.first[r], begin = sh.first[r] * HC + open_hc[h] * nt;
    c0[h] = cta_of(begin);
    c1[h] = cta_of(begin + nt - 1 - empty);
  }
  if (tid == 0) {
    __threadfence();  // the CTA's partial results (seen here by the barrier) before the count
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (open_row[h] >= 0) {
        const int before = atomicAdd(p.counters + c0[h], 1);
        sh.last[h] = before == c1[h] - c0[h];
        if (sh.last[h]) p.counters[c0[h]] = 0;  // nobody else comes: back to zero for the next call
      }
    __threadfence();
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (open_row[h] < 0 || !sh.last[h]) continue;
    const int count = c1[h] - c0[h] + 1;
    auto at = [&](int k) {
      return p.partials + ((int64_t)(c0[h] + k) * kPartialSlots + (k == 0 ? 1 : 0)) * partial_floats(DP);
    };
    int64_t h0;
    const int hn = columns(open_row[h], open_hc[h], h0);
    const int64_t row = (int64_t)p.row0 + open_row[h];
    for (int head = warp; head < hn; head += NW) {
      // 32 partial results at a time, lane j at the j-th; their m and l, and the first ones' elements, at once
      float top = -CUDART_INF_F, sum = 0.f;
      float4 acc[(DP + 127) / 128] = {};
      for (int k0 = 0; k0 < count; k0 += 32) {
        const int kn = min(32, count - k0);
        float m = -CUDART_INF_F, l = 0.f;
        if (lane < kn) {
          const float *x = at(k0 + lane) + kMaxGroup * DP + head;
          m = __ldcg(x), l = __ldcg(x + 16);
        }
        const float before = top;
        top = fmaxf(top, warp_max(m));
        const float base = top == -CUDART_INF_F ? 0.f : top, keep = exp2_fast(before - base);
        const float w = exp2_fast(m - base);
        sum = sum * keep + warp_sum(w * l);
#pragma unroll
        for (int i = 0; i < (DP + 127) / 128; ++i) {
          acc[i].x *= keep, acc[i].y *= keep, acc[i].z *= keep, acc[i].w *= keep;
          const int j = i * 32 + lane;
          const bool on = j < DP / 4;
#pragma unroll 16
          for (int k = 0; k < kn; ++k) {
            const float4 f = on ? __ldcg(reinterpret_cast<const float4 *>(at(k0 + k)) + head * (DP / 4) + j)
                                : make_float4(0.f, 0.f, 0.f, 0.f);
            const float x = __shfl_sync(~0u, w, k);
            acc[i].x += x * f.x, acc[i].y += x * f.y, acc[i].z += x * f.z, acc[i].w += x * f.w;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < (DP + 127) / 128; ++i) {
        if (!__any_sync(~0u, odd(acc[i]) != 0.f)) continue;
        acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i * 32 + lane >= DP / 4) continue;
#pragma unroll 1
        for (int k = 0; k < count; ++k) {
          const float m = __ldcg(at(k) + kMaxGroup * DP + head), base = top == -CUDART_INF_F ? 0.f : top;
          add_weighed(acc[i], exp2_fast(m - base),
                      __ldcg(reinterpret_cast<const float4 *>(at(k)) + head * (DP / 4) + i * 32 + lane));
        }
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
      for (int i = 0; i < (DP + 127) / 128; ++i) {
        acc[i].x *= inv, acc[i].y *= inv, acc[i].z *= inv, acc[i].w *= inv;
        const int j = i * 32 + lane;
        if (j < DP / 4 && j * 4 < D)
          *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + (row + below(head)) * a.ldo + (h0 + in(head)) * D +
                                     j * 4) = pack4(acc[i]);
      }
      if (a.lse && lane == 0) a.lse[(row + below(head)) * a.num_q_heads + h0 + in(head)] = lse_of(top, sum);
    }
  }
}

constexpr size_t kCounterBytes = 4096;
int attn_ctas() { return min(sm_count(), (int)(kCounterBytes / sizeof(int32_t))); }  // one per SM

template <int DT, int DP, int NB, bool PAGED16, bool PACK>
cudaError_t launch(const AttnParams &p, int32_t *status, cudaStream_t stream) {
  using Smem = AttnSmem<DP, attn_warps(DP), NB, PACK>;
  static_assert(sizeof(Smem) <= 227 * 1024, "fits in shared memory");
  cudaError_t e = raise_smem<kv_attention_kernel<DT, DP, NB, PAGED16, PACK>>((int)sizeof(Smem));
  if (e != cudaSuccess) return e;
  e = launch_waiting(kv_attention_kernel<DT, DP, NB, PAGED16, PACK>, dim3(attn_ctas()), dim3(attn_warps(DP) * 32),
                     sizeof(Smem), 1, stream, p, status);
  if (e == cudaSuccess) api_count_launch();
  return e;
}

template <int DT, int DP, bool PAGED16>
cudaError_t dispatch_columns(const AttnParams &p, int32_t *status, cudaStream_t stream) {
  const bool two = p.pack * p.group > 8;
  if (p.pack > 1)
    return two ? launch<DT, DP, 2, PAGED16, true>(p, status, stream) : launch<DT, DP, 1, PAGED16, true>(p, status, stream);
  if (two) return launch<DT, DP, 2, PAGED16, false>(p, status, stream);
  return launch<DT, DP, 1, PAGED16, false>(p, status, stream);
}
template <int DT, int DP>
cudaError_t dispatch(const AttnParams &p, int32_t *status, cudaStream_t stream) {
  return p.c.page_tokens % 16 == 0 ? dispatch_columns<DT, DP, true>(p, status, stream)
                                   : dispatch_columns<DT, DP, false>(p, status, stream);
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

bool kv_attention_fits(const mlora_kv_cache &c, const mlora_kv_attn &a) {
  const int64_t chunks = (a.num_q_heads / c.num_kv_heads + kMaxGroup - 1) / kMaxGroup;
  return ((int64_t)a.max_pages * c.page_tokens / 16 + 3) * c.num_kv_heads * chunks <= INT32_MAX;
}

int64_t kv_attention_workspace_bytes(int32_t head_dim) {
  const int dp = padded_dim(head_dim);
  return (int64_t)kCounterBytes + (int64_t)attn_ctas() * kPartialSlots * partial_floats(dp) * sizeof(float);
}

cudaError_t launch_kv_attention(const mlora_kv_cache &c, const mlora_kv_attn &a, int32_t layer, int32_t rows_per_request,
                                int32_t *status, cudaStream_t stream) {
  AttnParams p{};
  p.c = c;
  p.a = a;
  p.k = static_cast<const uint16_t *>(c.k) + layer * c.layer_stride;
  p.v = static_cast<const uint16_t *>(c.v) + layer * c.layer_stride;
  p.page = fast_div(c.page_tokens);
  p.group = a.num_q_heads / c.num_kv_heads;
  p.chunks = (p.group + kMaxGroup - 1) / kMaxGroup;
  const int64_t per_sm = a.num_rows * (int64_t)c.num_kv_heads / attn_ctas();
  // rows of a request: what the caller says (the most), or as many as the arrays have place for on average
  const int64_t most = rows_per_request ? rows_per_request
                                        : (a.num_rows + (int64_t)a.num_requests - 1) / std::max(1, a.num_requests);
  const int columns = per_sm >= kShare16 && most > 8 / p.group ? 16 : 8;
  p.pack = a.row_request && most > 1 && per_sm >= kShare8 ? std::max(1, columns / p.group) : 1;
  if (rows_per_request) p.pack = std::min(p.pack, rows_per_request);
  p.by_group = fast_div(p.group);
  p.scale_log2 = a.scale * 1.44269504088896340736f;
  p.counters = static_cast<int32_t *>(a.workspace);
  p.partials = reinterpret_cast<float *>(static_cast<char *>(a.workspace) + kCounterBytes);
  // rows of a launch: few enough that its tiles are counted in 31 bits, whatever the lengths (with kNone's empty ones)
  const int64_t row_tiles = ((int64_t)a.max_pages * c.page_tokens / 16 + 3) * c.num_kv_heads * p.chunks;
  const int32_t step = (int32_t)std::min<int64_t>(kRowsPerLaunch, INT32_MAX / row_tiles);
  if (step < 1) return cudaErrorInvalidValue;  // (refused before: kv_attention_fits)
  for (int64_t row0 = 0; row0 < a.num_rows; row0 += step) {  // (the last step may pass 2^31)
    p.row0 = (int32_t)row0;
    p.rows = (int32_t)std::min<int64_t>(step, a.num_rows - row0);
    const cudaError_t e = c.dtype == MLORA_BF16 ? dispatch<MLORA_BF16>(p, status, stream)
                                                : dispatch<MLORA_FP16>(p, status, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace mlora
