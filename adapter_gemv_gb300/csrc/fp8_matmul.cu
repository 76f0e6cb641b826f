// fp8_matmul.cu -- y = x W^T of e4m3 operands with a scale for each block of 128 (sm_103a).
//
//   y[i][n] = sum over blocks b of sx[i][b] sw[n / 128][b] p_b[i][n],   p_b = the products' sum over block b
//
// The tensor cores work out a block's p (four MMAs of K = 32, 128 rows of x by 128 columns) in one of two TMEM
// accumulators; warps read it back and add it, times its two scales, to sums in registers while the MMAs of the next block
// run in the other. A block of K is 128 bytes of a row: one row of the 128-byte swizzle.
//
// Few rows: W is read once, from memory, and that bounds; the MMAs' 128 rows are mostly empty then, and only the warps whose
// rows are there read back. The K blocks of a tile are split over a cluster of up to 8 CTAs, which
// add their sums through distributed shared memory in rank order.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "serve.cuh"
#include "tc.cuh"
#include "tensormap.h"

namespace mlora {

namespace {

constexpr int kRows = 128, kCols = 128, kBlock = MLORA_FP8_BLOCK;  // the MMA's tile; K bytes of a stage
constexpr int kThreads = 192;      // four warps of sums, a warp of loads, a warp of MMAs
constexpr int kMaxStages = 6;
constexpr int kMaxSplit = 8;
constexpr int kSmem = 111 * 1024;  // two CTAs an SM
constexpr int kHead = 1024;        // barriers, before the ring
constexpr int kSumLd = kCols + 4;  // floats of a row of sums in shared memory: lanes' 16-byte stores on different banks

struct MatmulParams {
  mlora_matmul a;
  int32_t mt, nt, blocks;  // tiles of rows, of columns; blocks of K
  int32_t box;             // rows of x that a stage holds
  int32_t stages, split;
};

struct Head {
  uint64_t full[kMaxStages], empty[kMaxStages], ready[2], taken[2];
  uint64_t drained;
  uint32_t tmem;
  int32_t late;
};
static_assert(sizeof(Head) <= kHead, "barriers fit");

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

template <int DT>
__global__ void __launch_bounds__(kThreads, 2) matmul_kernel(const __grid_constant__ MatmulParams p,
                                                             const __grid_constant__ CUtensorMap map_x,
                                                             const __grid_constant__ CUtensorMap map_w, int32_t *status) {
  extern __shared__ uint8_t raw[];
  uint8_t *smem = raw + (-smem_u32(raw) & 1023u);
  Head &sh = *reinterpret_cast<Head *>(smem);
  // The stages' x, then their W. An MMA reads 128 rows from where a stage's x begins: with fewer in the box those behind
  // belong to what follows, and their sums to rows that are not there.
  uint8_t *xring = smem + kHead, *wring = xring + p.stages * p.box * kBlock;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = p.split > 1 ? (int)cluster_ctarank() : 0;
  const int tile = blockIdx.x / p.split;
  const int m0 = tile % p.mt * kRows, nb = tile / p.mt;  // (CTAs of one tile of W are neighbours)
  const int rows = min(kRows, p.a.num_rows - m0);
  const int b0 = (int)((int64_t)p.blocks * c / p.split), b1 = (int)((int64_t)p.blocks * (c + 1) / p.split);
  const int warps = (rows + 31) / 32;  // that have rows

  if (tid == 0) {
    for (int s = 0; s < p.stages; ++s) mbar_init(&sh.full[s], 1), mbar_init(&sh.empty[s], 1);
    for (int s = 0; s < 2; ++s) mbar_init(&sh.ready[s], 1), mbar_init(&sh.taken[s], warps);
    mbar_init(&sh.drained, 1);
    sh.late = 0;
    mbar_fence_init();
    tc::tma_prefetch_desc(&map_x);
    tc::tma_prefetch_desc(&map_w);
  }
  if (warp == 5) tc::tmem_alloc(&sh.tmem, 2 * kCols);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = sh.tmem;
  pdl_wait();
  pdl_launch_dependents();

  float2 acc[kCols / 2];
  if (warp == 4) {
    if (lane == 0) {
      int i = 0;
      for (; i < b1 - b0; ++i) {
        const int s = i % p.stages;
        if (i >= p.stages && !mbar_wait(&sh.empty[s], (uint32_t)(i / p.stages - 1) & 1u)) {
          sh.late = 1;
          break;
        }
        mbar_arrive_expect_tx(&sh.full[s], (uint32_t)((kCols + p.box) * kBlock));
        tc::tma_load_2d(wring + s * kCols * kBlock, &map_w, (b0 + i) * kBlock, nb * kCols, &sh.full[s]);
        tc::tma_load_2d(xring + s * p.box * kBlock, &map_x, (b0 + i) * kBlock, m0, &sh.full[s]);
      }
      // nothing may land in shared memory after the CTA exits
      for (int k = max(i - p.stages, 0); k < i; ++k) (void)mbar_wait(&sh.full[k % p.stages], (uint32_t)(k / p.stages) & 1u, kDrainLimitNs);
    }
  } else if (warp == 5) {
    if (lane == 0) {
      constexpr uint32_t idesc = tc::idesc_e4m3(kRows, kCols);
      for (int i = 0; i < b1 - b0; ++i) {
        const int s = i % p.stages, t = i & 1;
        if ((i >= 2 && !mbar_wait(&sh.taken[t], (uint32_t)(i / 2 - 1) & 1u)) || !mbar_wait(&sh.full[s], (uint32_t)(i / p.stages) & 1u)) {
          sh.late = 1;
          break;
        }
        tc::tc_fence_after();
        const uint8_t *w = wring + s * kCols * kBlock, *x = xring + s * p.box * kBlock;
#pragma unroll
        for (int k = 0; k < kBlock / 32; ++k)
          tc::mma_f8(tmem + (uint32_t)(t * kCols), tc::smem_desc_sw128(x + k * 32, 16, 1024), tc::smem_desc_sw128(w + k * 32, 16, 1024),
                     idesc, k > 0);
        tc::mma_commit(&sh.empty[s]);
        tc::mma_commit(&sh.ready[t]);
      }
      tc::mma_commit(&sh.drained);
      (void)mbar_wait(&sh.drained, 0, kDrainLimitNs);
    }
  } else if (warp < warps) {
    const int row = min(m0 + tid, p.a.num_rows - 1);
    const float *sx = p.a.x_scale + row * p.a.ldxs, *sw = p.a.w_scale + nb * p.a.ldws;
#pragma unroll
    for (int j = 0; j < kCols / 2; ++j) acc[j] = make_float2(0.f, 0.f);
    float next_x = sx[b0], next_w = sw[b0];
    for (int i = 0; i < b1 - b0; ++i) {
      const int t = i & 1;
      const float s = next_x * next_w;
      if (i + 1 < b1 - b0) next_x = sx[b0 + i + 1], next_w = sw[b0 + i + 1];
      if (!mbar_wait(&sh.ready[t], (uint32_t)(i / 2) & 1u)) {
        sh.late = 1;
        break;
      }
      tc::tc_fence_after();
      const uint32_t at = tmem + ((uint32_t)(warp * 32) << 16) + (uint32_t)(t * kCols);
      const float2 ss = make_float2(s, s);
#pragma unroll
      for (int q = 0; q < kCols / 32; ++q) {
        uint32_t r[32];
        tc::tmem_ld32_async(at + q * 32, r);
        tc::tmem_ld_wait(r);
        if (q == kCols / 32 - 1) {
          tc::tc_fence_before();
          if (lane == 0) mbar_arrive(&sh.taken[t]);
        }
#pragma unroll
        for (int j = 0; j < 16; ++j)
          acc[q * 16 + j] = __ffma2_rn(ss, make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])), acc[q * 16 + j]);
      }
    }
  }
  // The ring is idle: every load has been multiplied, every product taken. It holds the tile's sums now.
  const bool late = __syncthreads_or(sh.late != 0);
  if (late) sh.late = 1;
  float *sums = reinterpret_cast<float *>(xring);
  if (!late && warp < 4 && tid < rows) {
#pragma unroll
    for (int j = 0; j < kCols / 4; ++j)
      *reinterpret_cast<float4 *>(sums + tid * kSumLd + j * 4) = make_float4(acc[2 * j].x, acc[2 * j].y, acc[2 * j + 1].x, acc[2 * j + 1].y);
  }
  tc::tc_fence_before();
  if (p.split > 1) cluster_sync();
  else __syncthreads();
  if (warp == 5) tc::tmem_dealloc(tmem, 2 * kCols);
  bool any_late = late;
  for (int k = 0; k < p.split && p.split > 1; ++k) any_late |= dsmem_ld_s32(dsmem_addr(&sh.late, k)) != 0;
  if (!any_late) {
    // chunks of 8 columns, shared out over the cluster
    const int all = rows * (kCols / 8), first = (int)((int64_t)all * c / p.split), end = (int)((int64_t)all * (c + 1) / p.split);
    for (int e = first + tid; e < end; e += kThreads) {
      const int i = e / (kCols / 8), n = e % (kCols / 8) * 8;
      if (nb * kCols + n >= p.a.d_out) continue;
      float v[8] = {};
      if (p.split == 1) {
        *reinterpret_cast<float4 *>(v) = *reinterpret_cast<const float4 *>(sums + i * kSumLd + n);
        *reinterpret_cast<float4 *>(v + 4) = *reinterpret_cast<const float4 *>(sums + i * kSumLd + n + 4);
      } else {
        for (int k = 0; k < p.split; ++k) {
          const uint32_t at = dsmem_addr(sums + i * kSumLd + n, k);
          const float4 a = dsmem_ld_f32x4(at), b = dsmem_ld_f32x4(at + 16);
          v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w, v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
        }
      }
      *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.a.y) + (int64_t)(m0 + i) * p.a.ldy + nb * kCols + n) = pack8<DT>(v);
    }
  } else if (tid == 0) {
    report(status, MLORA_STATUS_TIMEOUT);
  }
  if (p.split > 1) cluster_sync();  // a peer may still read these sums
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

template <int DT>
cudaError_t launch(MatmulParams p, int32_t *status, cudaStream_t stream) {
  const mlora_matmul &a = p.a;
  p.nt = (a.d_out - 1) / kCols + 1;
  p.mt = (a.num_rows - 1) / kRows + 1;
  p.blocks = (a.d_in - 1) / kBlock + 1;
  p.box = a.num_rows < kRows ? (a.num_rows + 7) & ~7 : kRows;
  const int64_t tiles = (int64_t)p.mt * p.nt;
  // K split until the CTAs fill the SMs, two each
  p.split = 1;
  while (p.split < kMaxSplit && tiles * p.split * 2 <= 2 * sm_count() && p.split * 2 <= p.blocks) p.split *= 2;
  const int stage = kCols * kBlock + p.box * kBlock;
  p.stages = std::min(kMaxStages, (kSmem - kHead - 1024) / stage);
  CUtensorMap map_x, map_w;
  if (!encode_bytes(&map_x, a.x, a.d_in, a.num_rows, a.ldx, p.box) || !encode_bytes(&map_w, a.w, a.d_in, a.d_out, a.ldw, kCols))
    return cudaErrorInvalidValue;
  cudaError_t e = raise_smem<matmul_kernel<DT>>(kSmem);
  if (e != cudaSuccess) return e;
  e = launch_waiting(matmul_kernel<DT>, dim3((unsigned)(tiles * p.split)), dim3(kThreads), kSmem, p.split, stream, p, map_x, map_w, status);
  if (e == cudaSuccess) api_count_launch();
  return e;
}

}  // namespace

cudaError_t launch_fp8_matmul(const mlora_matmul &a, int32_t *status, cudaStream_t stream) {
  // rows of a launch: its tiles are counted in 31 bits, eight times over
  const int64_t most = std::max<int64_t>(1, (INT32_MAX / kMaxSplit) / ((a.d_out - 1) / kCols + 1)) * kRows;
  for (int64_t row0 = 0; row0 < a.num_rows; row0 += most) {
    MatmulParams p{};
    p.a = a;
    p.a.num_rows = (int32_t)std::min<int64_t>(most, a.num_rows - row0);
    p.a.x = static_cast<const uint8_t *>(a.x) + row0 * a.ldx;
    p.a.x_scale = a.x_scale + row0 * a.ldxs;
    p.a.y = static_cast<uint16_t *>(a.y) + row0 * a.ldy;
    const cudaError_t e = a.dtype == MLORA_BF16 ? launch<MLORA_BF16>(p, status, stream) : launch<MLORA_FP16>(p, status, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace mlora
