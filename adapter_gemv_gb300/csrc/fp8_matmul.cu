// fp8_matmul.cu -- y = x W^T of e4m3 operands with a scale for each block of 128 (sm_103a).
//
//   y[i][n] = sum over blocks b of sx[i][b] sw[n / 128][b] p_b[i][n],   p_b = the products' sum over block b
//
// The tensor cores work out a block's p (four MMAs of K = 32) in one of two or four TMEM accumulators; warps read it
// back and add it, times its two scales, to sums in registers while the MMAs of the next blocks run in the others. A block of
// K is 128 bytes of a row: one row of the 128-byte swizzle, so a TMA box is an operand of the MMA as it lies. The sums are in
// fp32, the blocks in order, and rounded once.
//
// Few rows: W is read once, from memory, and that bounds. W's rows are the MMA's 128, x's its 16, 32 or 64 columns, so a product
// is read back with 16 to 64 values a lane. The K blocks of a tile are split over a cluster of up to 8 CTAs, which add
// their sums through distributed shared memory in rank order. 32 x 4096 x 22016 (92 MB): 17.8 us, 5.2 TB/s (20 SMs of 152
// have two tiles); 8 x 8192 x 28672 38.0 us, 6.2 TB/s; 1 x 4096 x 4096 5.8 us.
//
// Many rows: 128 of x by up to 256 of W, one persistent CTA an SM. 12604 x 5120 x 13824: 815 to 835 us, 2.15 PFLOP/s. Bound by the
// length of a turn: a tile's block is 32768 sums, 256 cycles of the SM's FMA units, and its MMAs take 512 in the other accumulator
// meanwhile, but a turn takes 1000: a warp reads its part of TMEM 8 columns at a time, eight trips one behind the other, with one
// on its way at any moment. (2048 x 4096 x 11008 under ncu: tensor cores 41 % busy, FMA units 25 %, schedulers 59 %; most stalls
// are such waits.) Tried on 7680 x 8192 x 7680 (353 us then, 375 to 410 by the card's clock): a pair of CTAs on 256 rows
// (cta_group::2, half the loads of W) 4 % slower; four accumulators of 128 columns 17 %; the next turn's barrier polled
// early 6 %; loads of 16 and 32 columns at a time spill and are slower.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "serve.cuh"
#include "tc.cuh"
#include "tensormap.h"

namespace mlora {

namespace {

constexpr int kTile = 128, kBlock = MLORA_FP8_BLOCK;  // the MMA's rows a CTA; K bytes of a stage
constexpr int kChunk = 8;                             // blocks whose scales are brought together

struct MatmulParams {
  mlora_matmul a;
  int32_t mt, nt, blocks;  // tiles of x's rows, of W's; blocks of K
  int32_t cols;            // many rows: W's rows of a tile
  int32_t split;           // few rows: CTAs that share a tile's blocks
  int32_t stages;
  uint64_t wait_ns;        // limit of a wait
};

__device__ __forceinline__ float4 dsmem_ld_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ int32_t dsmem_ld_s32(uint32_t addr) {
  int32_t v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// An arrival that orders no memory: what it hands over, accumulators that have been read, is ordered by the tcgen05 fences. A
// release waits for the thread's memory accesses in flight (between two CTAs that doubled a block's time).
__device__ __forceinline__ void mbar_arrive_relaxed(uint32_t addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

__device__ __forceinline__ float lds_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// Where in the ring, and whether it is an odd time around.
struct Turn {
  int at = 0;
  uint32_t odd = 0;
  __device__ __forceinline__ void next(int n) {
    if (++at == n) at = 0, odd ^= 1;
  }
};

// Behind its last load, the warp of loads waits until all have landed, whichever warp gave up before it used them: a CTA ends
// with none on its way. `turn`: the next load's; a stage that had none is through its wait at once.
__device__ __forceinline__ void drain_loads(uint64_t *full, const Turn &turn, int stages) {
  for (int s = 0; s < stages; ++s) (void)tc::mbar_wait_warp<false>(&full[s], s < turn.at ? turn.odd : turn.odd ^ 1u, kDrainLimitNs);
}
// The same of the warp of MMAs: none is at work on shared memory or TMEM when the CTA gives them up.
__device__ __forceinline__ void drain_mmas(uint64_t *drained) {
  if (tc::elect_one()) tc::mma_commit(drained);
  __syncwarp();
  (void)tc::mbar_wait_warp<false>(drained, 0, kDrainLimitNs);
}

// ---- few rows: 128 rows of W (the MMA's M) by NT rows of x ----------------------------------------------------

constexpr int kFewThreads = 256;      // four warps of sums, a warp of loads, a warp of MMAs, two warps of scales
constexpr int kFewStages = 8;
constexpr int kMaxSplit = 8;
constexpr int kFewSmem = 111 * 1024;  // two CTAs an SM
constexpr int kFewHead = 5 * 1024;
constexpr int kSumLd = kTile + 4;     // floats of a row of sums in shared memory

template <int NT>
struct FewHead {
  static constexpr int kBufs = 4;  // accumulators in TMEM
  uint64_t full[kFewStages], empty[kFewStages], ready[kBufs], taken[kBufs], scaled[2], used[2];
  uint64_t drained;
  uint32_t tmem;
  int32_t late;
  alignas(16) float sx[2 * kChunk][NT];  // two chunks
  float sw[2 * kChunk];
};

template <int DT, int NT, bool SHORT>
__global__ void __launch_bounds__(kFewThreads, 2) few_rows_kernel(const __grid_constant__ MatmulParams p,
                                                                  const __grid_constant__ CUtensorMap map_x,
                                                                  const __grid_constant__ CUtensorMap map_w, int32_t *status) {
  using Head = FewHead<NT>;
  constexpr int kBufs = Head::kBufs, kTmem = kBufs * NT;
  static_assert(sizeof(Head) <= kFewHead, "barriers and scales fit");
  extern __shared__ uint8_t raw[];
  uint8_t *smem = raw + (-smem_u32(raw) & 1023u);
  Head &sh = *reinterpret_cast<Head *>(smem);
  uint8_t *wring = smem + kFewHead, *xring = wring + p.stages * kTile * kBlock;
  const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;
  const int c = p.split > 1 ? (int)cluster_ctarank() : 0;
  const int tile = blockIdx.x / p.split;
  const int m0 = tile % p.mt * NT, nb = tile / p.mt;  // (CTAs of one tile of W are neighbours)
  const int rows = min(NT, p.a.num_rows - m0);
  const int b0 = (int)((int64_t)p.blocks * c / p.split), n_blocks = (int)((int64_t)p.blocks * (c + 1) / p.split) - b0;

  if (tid == 0) {
    for (int s = 0; s < p.stages; ++s) mbar_init(&sh.full[s], 1), mbar_init(&sh.empty[s], 1);
    for (int s = 0; s < kBufs; ++s) mbar_init(&sh.ready[s], 1), mbar_init(&sh.taken[s], 4);
    for (int s = 0; s < 2; ++s) mbar_init(&sh.scaled[s], 64), mbar_init(&sh.used[s], 4);
    mbar_init(&sh.drained, 1);
    sh.late = 0;
    mbar_fence_init();
    tc::tma_prefetch_desc(&map_x);
    tc::tma_prefetch_desc(&map_w);
  }
  if (warp == 5) tc::tmem_alloc(&sh.tmem, kTmem);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = sh.tmem;
  pdl_wait();
  pdl_launch_dependents();

  float acc[NT];
  bool gone = false;
  // (The warps of loads and of MMAs wait as a whole and elect the lane that issues: alone in a branch, a lane's poll of a
  // barrier takes 160 cycles instead of 50.)
  if (warp == 4) {
    Turn turn;
    for (int i = 0; i < n_blocks; ++i, turn.next(p.stages)) {
      const int s = turn.at;
      if (!tc::mbar_wait_warp<SHORT>(&sh.empty[s], turn.odd ^ 1u, p.wait_ns)) {
        gone = true;
        break;
      }
      if (tc::elect_one()) {
        mbar_arrive_expect_tx(&sh.full[s], (uint32_t)((kTile + NT) * kBlock));
        tc::tma_load_2d(wring + s * kTile * kBlock, &map_w, (b0 + i) * kBlock, nb * kTile, &sh.full[s]);
        tc::tma_load_2d(xring + s * NT * kBlock, &map_x, (b0 + i) * kBlock, m0, &sh.full[s]);
      }
      __syncwarp();
    }
    if (gone) sh.late = 1;
    drain_loads(sh.full, turn, p.stages);
  } else if (warp == 5) {
    constexpr uint32_t idesc = tc::idesc_e4m3(kTile, NT);
    Turn turn, buf;
    for (int i = 0; i < n_blocks; ++i, turn.next(p.stages), buf.next(kBufs)) {
      const int s = turn.at;
      if (!tc::mbar_wait_warp<SHORT>(&sh.taken[buf.at], buf.odd ^ 1u, p.wait_ns) || !tc::mbar_wait_warp<SHORT>(&sh.full[s], turn.odd, p.wait_ns)) {
        gone = true;
        break;
      }
      tc::tc_fence_after();
      if (tc::elect_one()) {
        const uint8_t *w = wring + s * kTile * kBlock, *x = xring + s * NT * kBlock;
#pragma unroll
        for (int k = 0; k < kBlock / 32; ++k)
          tc::mma_f8(tmem + (uint32_t)(buf.at * NT), tc::smem_desc_sw128(w + k * 32, 16, 1024), tc::smem_desc_sw128(x + k * 32, 16, 1024),
                     idesc, k > 0);
        tc::mma_commit(&sh.ready[buf.at]);
        tc::mma_commit(&sh.empty[s]);
      }
      __syncwarp();
    }
    if (gone) sh.late = 1;
    drain_mmas(&sh.drained);
  } else if (warp >= 6) {
    // scales, kChunk blocks at a time: thread i those of x's row i, and of W's rows block i of them
    const int i = tid - 6 * 32;
    const float *sx = p.a.x_scale + (int64_t)min(m0 + i, p.a.num_rows - 1) * p.a.ldxs + b0;
    const float *sw = p.a.w_scale + nb * p.a.ldws + b0;
    Turn chunk;
    for (int b = 0; b < n_blocks; b += kChunk, chunk.next(2)) {
      float v[kChunk] = {};
#pragma unroll
      for (int k = 0; k < kChunk; ++k)
        if (i < NT && b + k < n_blocks) v[k] = sx[b + k];
      const float w = i < kChunk && b + i < n_blocks ? sw[b + i] : 0.f;
      if (!tc::mbar_wait_warp<SHORT>(&sh.used[chunk.at], chunk.odd ^ 1u, p.wait_ns)) {
        sh.late = 1;
        break;
      }
#pragma unroll
      for (int k = 0; k < kChunk; ++k)
        if (i < NT) sh.sx[chunk.at * kChunk + k][i] = v[k];
      if (i < kChunk) sh.sw[chunk.at * kChunk + i] = w;
      mbar_arrive(&sh.scaled[chunk.at]);
    }
  } else {
    // a thread a row of W
    const uint32_t taken0 = dsmem_addr(sh.taken, c);
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j] = 0.f;
    Turn buf, chunk;
    for (int i = 0; i < n_blocks; ++i) {
      if (i % kChunk == 0 && !tc::mbar_wait_warp<SHORT>(&sh.scaled[chunk.at], chunk.odd, p.wait_ns)) gone = true;
      const float *sx = sh.sx[chunk.at * kChunk + i % kChunk];
      const float sw = sh.sw[chunk.at * kChunk + i % kChunk];
      if (gone || !tc::mbar_wait_warp<SHORT>(&sh.ready[buf.at], buf.odd, p.wait_ns)) {
        gone = true;
        break;
      }
      tc::tc_fence_after();
      const uint32_t at = tmem + ((uint32_t)(warp * 32) << 16) + (uint32_t)(buf.at * NT);
      // 8 columns are added while the next 8 are on their way
      uint32_t r[2][8];
      tc::tmem_ld8_async(at, r[0]);
#pragma unroll
      for (int q = 0; q < NT / 8; ++q) {
        tc::tmem_ld_wait(r[q & 1]);
        if (q < NT / 8 - 1) {
          tc::tmem_ld8_async(at + (q + 1) * 8, r[(q + 1) & 1]);
        } else {
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_relaxed(taken0 + buf.at * 8);
        }
        const float4 a = *reinterpret_cast<const float4 *>(sx + q * 8), b = *reinterpret_cast<const float4 *>(sx + q * 8 + 4);
        const float s[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[q * 8 + j] = fmaf(s[j] * sw, __uint_as_float(r[q & 1][j]), acc[q * 8 + j]);
      }
      buf.next(kBufs);
      if (i % kChunk == kChunk - 1 || i == n_blocks - 1) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.used[chunk.at]);
        chunk.next(2);
      }
    }
    if (gone) sh.late = 1;
  }
  // The ring is idle: every load has been multiplied, every product taken. It holds the tile's sums now.
  const bool late = __syncthreads_or(sh.late != 0);
  if (late) sh.late = 1;
  float *sums = reinterpret_cast<float *>(wring);
  if (!late && warp < 4) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
      if (j < rows) sums[j * kSumLd + tid] = acc[j];
  }
  tc::tc_fence_before();
  if (p.split > 1) cluster_sync();
  else __syncthreads();
  if (warp == 5) tc::tmem_dealloc(tmem, kTmem);
  bool any_late = late;
  for (int k = 0; k < p.split && p.split > 1; ++k) any_late |= dsmem_ld_s32(dsmem_addr(&sh.late, k)) != 0;
  if (!any_late) {
    // chunks of 8 columns, shared out over the cluster
    const int all = rows * (kTile / 8), first = all * c / p.split, end = all * (c + 1) / p.split;
    for (int e = first + tid; e < end; e += kFewThreads) {
      const int i = e / (kTile / 8), n = e % (kTile / 8) * 8;
      if (nb * kTile + n >= p.a.d_out) continue;
      float v[8] = {};
      if (p.split == 1) {
        *reinterpret_cast<float4 *>(v) = *reinterpret_cast<const float4 *>(sums + i * kSumLd + n);
        *reinterpret_cast<float4 *>(v + 4) = *reinterpret_cast<const float4 *>(sums + i * kSumLd + n + 4);
      } else {
        float4 a[kMaxSplit], b[kMaxSplit];  // all on their way before the first is added
#pragma unroll
        for (int k = 0; k < kMaxSplit; ++k)
          if (k < p.split) {
            const uint32_t at = dsmem_addr(sums + i * kSumLd + n, k);
            a[k] = dsmem_ld_f32x4(at), b[k] = dsmem_ld_f32x4(at + 16);
          }
#pragma unroll
        for (int k = 0; k < kMaxSplit; ++k)
          if (k < p.split)
            v[0] += a[k].x, v[1] += a[k].y, v[2] += a[k].z, v[3] += a[k].w, v[4] += b[k].x, v[5] += b[k].y, v[6] += b[k].z, v[7] += b[k].w;
      }
      *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.a.y) + (int64_t)(m0 + i) * p.a.ldy + nb * kTile + n) = pack8<DT>(v);
    }
  } else if (tid == 0) {
    report(status, MLORA_STATUS_TIMEOUT);
  }
  if (p.split > 1) cluster_sync();  // a peer may still read these sums
}

// ---- many rows: 128 rows of x by up to 256 rows of W ---------------------------------------------------------

constexpr int kManyThreads = 640;  // sixteen warps of sums, a warp of loads, a warp of MMAs, two warps of scales
constexpr int kManyStages = 7;
constexpr int kManySmem = 227 * 1024;
constexpr int kManyHead = 10 * 1024;
constexpr int kMaxCols = 256;  // columns of a tile: two accumulators of them fill the TMEM

struct ManyHead {
  uint64_t full[kManyStages], empty[kManyStages], ready[2], taken[2], scaled[2], used[2];
  uint64_t drained;
  uint32_t tmem;
  int32_t late;
  float sx[2 * kChunk][kTile], sw[2 * kChunk][kMaxCols / 32];  // two chunks; W's for each 32 of the tile's columns
};
static_assert(sizeof(ManyHead) <= kManyHead, "barriers and scales fit");

// Tile t of mt x nt: bands of kBand row tiles, in a band column by column, so that the tiles of one moment share
// rows of x and of W in L2.
constexpr int kBand = 8;
__device__ __forceinline__ void tile_at(const MatmulParams &p, int t, int &m, int &n) {
  const int band = t / (kBand * p.nt), in = t - band * kBand * p.nt;
  const int height = min(kBand, p.mt - band * kBand);
  n = in / height;
  m = band * kBand + in - n * height;
}

template <int DT, bool SHORT>
__global__ void __launch_bounds__(kManyThreads, 1) many_rows_kernel(const __grid_constant__ MatmulParams p,
                                                                    const __grid_constant__ CUtensorMap map_x,
                                                                    const __grid_constant__ CUtensorMap map_w, int32_t *status) {
  extern __shared__ uint8_t raw[];
  uint8_t *smem = raw + (-smem_u32(raw) & 1023u);
  ManyHead &sh = *reinterpret_cast<ManyHead *>(smem);
  const uint32_t stage_bytes = (uint32_t)((kTile + p.cols) * kBlock);
  uint8_t *ring = smem + kManyHead;
  const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;
  const int tiles = p.mt * p.nt;

  if (tid == 0) {
    for (int s = 0; s < p.stages; ++s) mbar_init(&sh.full[s], 1), mbar_init(&sh.empty[s], 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sh.ready[s], 1), mbar_init(&sh.taken[s], 16);
      mbar_init(&sh.scaled[s], 64), mbar_init(&sh.used[s], 16);
    }
    mbar_init(&sh.drained, 1);
    sh.late = 0;
    mbar_fence_init();
    tc::tma_prefetch_desc(&map_x);
    tc::tma_prefetch_desc(&map_w);
  }
  if (warp == 17) tc::tmem_alloc(&sh.tmem, 2 * kMaxCols);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = sh.tmem;
  pdl_wait();
  pdl_launch_dependents();

  // (The warps of loads and of MMAs wait as a whole and elect the lane that issues: alone in a branch, a lane's poll of a barrier
  // takes 160 cycles instead of 50.)
  if (warp == 16) {
    Turn turn;
    bool gone = false;
    for (int t = blockIdx.x; t < tiles && !gone; t += gridDim.x) {
      int m, n;
      tile_at(p, t, m, n);
      const int x0 = m * kTile, w0 = n * p.cols;
      for (int b = 0; b < p.blocks; ++b, turn.next(p.stages)) {
        const int s = turn.at;
        if (!tc::mbar_wait_warp<SHORT>(&sh.empty[s], turn.odd ^ 1u, p.wait_ns)) {
          gone = true;
          break;
        }
        if (tc::elect_one()) {
          uint8_t *at = ring + s * stage_bytes;
          mbar_arrive_expect_tx(&sh.full[s], stage_bytes);
          tc::tma_load_2d(at, &map_x, b * kBlock, x0, &sh.full[s]);
          tc::tma_load_2d(at + kTile * kBlock, &map_w, b * kBlock, w0, &sh.full[s]);
        }
        __syncwarp();
      }
    }
    if (gone) sh.late = 1;
    drain_loads(sh.full, turn, p.stages);
  } else if (warp == 17) {
    const uint32_t idesc = tc::idesc_e4m3(kTile, p.cols);
    Turn turn, acc;
    bool gone = false;
    for (int t = blockIdx.x; t < tiles && !gone; t += gridDim.x) {
      for (int b = 0; b < p.blocks; ++b, turn.next(p.stages), acc.next(2)) {
        const int s = turn.at;
        if (!tc::mbar_wait_warp<SHORT>(&sh.taken[acc.at], acc.odd ^ 1u, p.wait_ns) || !tc::mbar_wait_warp<SHORT>(&sh.full[s], turn.odd, p.wait_ns)) {
          gone = true;
          break;
        }
        tc::tc_fence_after();
        if (tc::elect_one()) {
          const uint8_t *x = ring + s * stage_bytes, *w = x + kTile * kBlock;
#pragma unroll
          for (int k = 0; k < kBlock / 32; ++k) {
            const uint64_t dx = tc::smem_desc_sw128(x + k * 32, 16, 1024), dw = tc::smem_desc_sw128(w + k * 32, 16, 1024);
            tc::mma_f8(tmem + (uint32_t)(acc.at * kMaxCols), dx, dw, idesc, k > 0);
          }
          tc::mma_commit(&sh.ready[acc.at]), tc::mma_commit(&sh.empty[s]);
        }
        __syncwarp();
      }
    }
    if (gone) sh.late = 1;
    drain_mmas(&sh.drained);
  } else if (warp >= 18) {
    // scales, kChunk blocks at a time, so that the sums read them from shared memory: from global memory, a row of x a
    // lane, they would be 32 sectors for each of 16 warps and every block
    const int i = tid - 18 * 32;
    Turn chunk;
    bool gone = false;
    for (int t = blockIdx.x; t < tiles && !gone; t += gridDim.x) {
      int m, n;
      tile_at(p, t, m, n);
      const int last = p.a.num_rows - 1, x0 = m * kTile;
      const float *xa = p.a.x_scale + min((int64_t)x0 + i, (int64_t)last) * p.a.ldxs, *xb = p.a.x_scale + min((int64_t)x0 + 64 + i, (int64_t)last) * p.a.ldxs;
      // W's: thread i brings block i / 8 of the chunk, columns i % 8 * 32 (a group of 32 lies in one block of W's rows)
      const float *wa = p.a.w_scale + min((int64_t)n * p.cols + i % 8 * 32, (int64_t)p.a.d_out - 1) / kBlock * p.a.ldws;
      for (int b = 0; b < p.blocks; b += kChunk, chunk.next(2)) {
        float va[kChunk], vb[kChunk];
#pragma unroll
        for (int k = 0; k < kChunk; ++k) {
          va[k] = b + k < p.blocks ? xa[b + k] : 0.f;
          vb[k] = b + k < p.blocks ? xb[b + k] : 0.f;
        }
        const float w = b + i / 8 < p.blocks ? wa[b + i / 8] : 0.f;
        if (!tc::mbar_wait_warp<SHORT>(&sh.used[chunk.at], chunk.odd ^ 1u, p.wait_ns)) {
          gone = true, sh.late = 1;
          break;
        }
#pragma unroll
        for (int k = 0; k < kChunk; ++k) sh.sx[chunk.at * kChunk + k][i] = va[k], sh.sx[chunk.at * kChunk + k][64 + i] = vb[k];
        sh.sw[chunk.at * kChunk + i / 8][i % 8] = w;
        mbar_arrive(&sh.scaled[chunk.at]);
      }
    }
  } else {
    // A thread a row of x (of the warp's quarter of the lanes), 64 of the tile's columns. 640 threads leave 96 registers each:
    // what the loop keeps beside the 64 sums and the 16 products on their way is kept small (the sums' spills, more than the L1
    // that 227 KB of shared memory leave, took twice the time).
    const int c0 = (warp >> 2) * 64;
    const uint32_t taken0 = dsmem_addr(sh.taken, 0), lanes = tmem + ((uint32_t)(warp & 3) << 21) + (uint32_t)c0;
    const uint32_t scale = smem_u32(&sh.sx[0][(warp & 3) * 32 + lane]), wscale = smem_u32(&sh.sw[0][c0 / 32]);
    uint32_t done = 0, chunks = 0;  // products and chunks of scales so far
    bool gone = false;
    for (int t = blockIdx.x; t < tiles && !gone; t += gridDim.x) {
      float acc[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) acc[j] = 0.f;
      for (int b = 0; b < p.blocks; ++b) {
        if (b % kChunk == 0) {
          if (!tc::mbar_wait_warp<SHORT>(&sh.scaled[chunks & 1], (chunks >> 1) & 1, p.wait_ns)) gone = true;
          ++chunks;
        }
        const int place = (int)((chunks - 1) & 1) * kChunk + b % kChunk;
        const float fx = lds_f32(scale + place * kTile * 4);
        const float f0 = fx * lds_f32(wscale + place * (kMaxCols / 8)), f1 = fx * lds_f32(wscale + place * (kMaxCols / 8) + 4);
        if (gone || !tc::mbar_wait_warp<SHORT>(&sh.ready[done & 1], (done >> 1) & 1, p.wait_ns)) {
          gone = true, sh.late = 1;
          break;
        }
        tc::tc_fence_after();
        const uint32_t at = lanes + (done & 1) * kMaxCols;
        // 8 columns are added while the next 8 are on their way (columns behind a narrower tile's are read as they are and not used)
        uint32_t r[2][8];
        tc::tmem_ld8_async(at, r[0]);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          tc::tmem_ld_wait(r[q & 1]);
          if (q < 7) {
            tc::tmem_ld8_async(at + (q + 1) * 8, r[(q + 1) & 1]);
          } else {
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_relaxed(taken0 + (done & 1) * 8);
            ++done;
          }
          const float f = q < 4 ? f0 : f1;
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[q * 8 + j] = fmaf(f, __uint_as_float(r[q & 1][j]), acc[q * 8 + j]);
        }
        if (b % kChunk == kChunk - 1 || b == p.blocks - 1) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.used[(chunks - 1) & 1]);
        }
      }
      int m, n;
      tile_at(p, t, m, n);
      const int64_t row = (int64_t)m * kTile + (warp & 3) * 32 + lane;
      const int n0 = n * p.cols + c0;
      if (gone || row >= p.a.num_rows) continue;
      uint16_t *y = static_cast<uint16_t *>(p.a.y) + row * p.a.ldy + n0;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = acc[q * 8 + j];
        if (c0 + q * 8 < p.cols && n0 + q * 8 < p.a.d_out) *reinterpret_cast<uint4 *>(y + q * 8) = pack8<DT>(v);
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (tid == 0 && sh.late) report(status, MLORA_STATUS_TIMEOUT);
  if (warp == 17) tc::tmem_dealloc(tmem, 2 * kMaxCols);
}

// Map of `rows` rows of `cols` bytes, ld apart; boxes of a block's 128 bytes by box_rows rows, zeros outside.
bool encode_bytes(CUtensorMap *m, const void *base, int64_t cols, int64_t rows, int64_t ld, int box_rows) {
  EncodeFn fn = encoder();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld};
  const cuuint32_t box[2] = {kBlock, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DT, int NT, bool SHORT>
cudaError_t launch_few(MatmulParams p, int32_t *status, cudaStream_t stream) {
  const mlora_matmul &a = p.a;
  p.nt = (a.d_out - 1) / kTile + 1;
  p.mt = (a.num_rows - 1) / NT + 1;
  p.stages = std::min(kFewStages, (kFewSmem - kFewHead - 1023) / ((kTile + NT) * kBlock));
  CUtensorMap map_x, map_w;
  if (!encode_bytes(&map_x, a.x, a.d_in, a.num_rows, a.ldx, NT) || !encode_bytes(&map_w, a.w, a.d_in, a.d_out, a.ldw, kTile))
    return cudaErrorInvalidValue;
  cudaError_t e = raise_smem<few_rows_kernel<DT, NT, SHORT>>(kFewSmem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((int64_t)p.mt * p.nt * p.split));
  e = launch_waiting(few_rows_kernel<DT, NT, SHORT>, grid, dim3(kFewThreads), kFewSmem, p.split, stream, p, map_x, map_w, status);
  if (e == cudaSuccess) api_count_launch();
  return e;
}

template <int DT, bool SHORT>
cudaError_t launch_many(MatmulParams p, int32_t *status, cudaStream_t stream) {
  const mlora_matmul &a = p.a;
  p.nt = (a.d_out - 1) / p.cols + 1;
  p.mt = (a.num_rows - 1) / kTile + 1;
  p.stages = std::min(kManyStages, (kManySmem - kManyHead - 1023) / ((kTile + p.cols) * kBlock));
  CUtensorMap map_x, map_w;
  if (!encode_bytes(&map_x, a.x, a.d_in, a.num_rows, a.ldx, kTile) || !encode_bytes(&map_w, a.w, a.d_in, a.d_out, a.ldw, p.cols))
    return cudaErrorInvalidValue;
  cudaError_t e = raise_smem<many_rows_kernel<DT, SHORT>>(kManySmem);
  if (e != cudaSuccess) return e;
  const dim3 grid(std::min(p.mt * p.nt, sm_count()));
  e = launch_waiting(many_rows_kernel<DT, SHORT>, grid, dim3(kManyThreads), kManySmem, 1, stream, p, map_x, map_w, status);
  if (e == cudaSuccess) api_count_launch();
  return e;
}

// SHORT: a limit of the waits that the caller has set.
template <int DT, bool SHORT>
cudaError_t dispatch(MatmulParams p, int32_t *status, cudaStream_t stream) {
  const int rows = p.a.num_rows, sms = sm_count();
  p.blocks = (p.a.d_in - 1) / kBlock + 1;
  // Few rows where its tiles (and there are up to 64 rows in one) leave no SM two of them: 128 x 4096 x 4096 10.0 us against 15.8,
  // 512 x 4096 x 1024 9.9 against 16.1; 213 x 8192 x 8192, 256 tiles: 33 against 30. And up to 64 rows in any case: 64 x 8192 x
  // 28672 42.3 against 41.5, 64 x 4096 x 11008 14.1 against 17.0.
  const int nt = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
  const int64_t tiles = (int64_t)((rows - 1) / nt + 1) * ((p.a.d_out - 1) / kTile + 1);
  if (rows <= 64 || tiles <= sms) {
    // K split as long as every CTA has an SM to itself: 1 x 4096 x 4096 9.6, 6.9, 5.3, 5.6 us with 1, 2, 4, 8 (256 CTAs); 64 rows of
    // it 12.6, 9.3, 8.1, 11.5; 1 x 4096 x 1024 9.6, 6.8, 5.0, 4.3
    p.split = (int)std::max<int64_t>(1, std::min<int64_t>(std::min(kMaxSplit, p.blocks), sms / tiles));
    if (nt == 16) return launch_few<DT, 16, SHORT>(p, status, stream);
    if (nt == 32) return launch_few<DT, 32, SHORT>(p, status, stream);
    return launch_few<DT, 64, SHORT>(p, status, stream);
  }
  // The width of the tiles by what the SM with the most of them takes: a block of K takes 600 + columns (0.42 us with 128,
  // 0.45 with 192, 0.5 with 256). 1024 x 8192 x 28672 with 128, 192, 224, 256 columns: 326, 232, 209, 198 us; 213 x 8192 x 28672 85,
  // 61, 64, 67; 1024 x 4096 x 4096 33, 36, 20, 21.
  int64_t least = INT64_MAX;
  const int64_t mt = (rows - 1) / kTile + 1;
  for (int cols = kMaxCols; cols >= 64; cols -= 32) {
    const int64_t most = (mt * ((p.a.d_out - 1) / cols + 1) + sms - 1) / sms, cost = most * (600 + cols);
    if (cost < least) least = cost, p.cols = cols;
  }
  return launch_many<DT, SHORT>(p, status, stream);
}

}  // namespace

// Tiles of 16 rows by 128 are counted in 31 bits, eight times over.
bool fp8_matmul_fits(const mlora_matmul &a) {
  return ((a.num_rows - 1) / 16 + 1) * (int64_t)((a.d_out - 1) / kTile + 1) <= INT32_MAX / kMaxSplit;
}

cudaError_t launch_fp8_matmul(const mlora_matmul &a, int32_t *status, uint64_t wait_ns, cudaStream_t stream) {
  MatmulParams p{};
  p.a = a;
  p.wait_ns = wait_ns ? wait_ns : kWaitLimitNs;
  const auto run = a.dtype == MLORA_BF16 ? (wait_ns ? dispatch<MLORA_BF16, true> : dispatch<MLORA_BF16, false>)
                                         : (wait_ns ? dispatch<MLORA_FP16, true> : dispatch<MLORA_FP16, false>);
  return run(p, status, stream);
}

}  // namespace mlora
