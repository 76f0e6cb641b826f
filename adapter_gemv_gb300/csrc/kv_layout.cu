// kv_layout.cu -- a step's places in the paged key-value cache, from the requests' lengths (sm_103a).
//
// With len and n a request's cached and new tokens, pt the tokens of a page and c(x) = ceil(x / pt):
//   rows    R_r = sum_{s<r} max(n_s, 0)          first row of request r
//   pages   P_r = sum_{s<r} c(len_s + n_s) - c(len_s)   (n_s >= 0)   first ring entry it pops
//   returns B_r = sum_{s<r} c(len_s)             (n_s < 0)    first ring entry it pushes
// Three exclusive sums over at most 8192 requests, after which every new page table entry, pushed page
// and row is a function of its index: entry j belongs to the request found by bisecting the sums.
//
// A few thousand whole numbers: the time is the chain launch -> lengths -> sums -> page ids ->
// stores. So one launch: a cluster of CTAs (one, when there is little to write) in which every CTA
// forms the same sums in its own shared memory, and the entries are dealt over the cluster's threads.
// kv_len_out and free_state_out may be the inputs: they are written behind a cluster barrier that
// every CTA reaches after its last read of those. Ring entries popped and pushed, and page table entries
// read and written, are different ones (popped: free before the call; pushed: behind those).
#include <cuda_runtime.h>
#include <stdint.h>

#include "serve.cuh"

namespace mlora {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

struct LayoutSmem {  // before the arrays [num_requests + 1] each: rows, pages, back, then len
  int64_t warp[3][kWarps];
  int64_t total[3];
};

// Largest r in [0, n) with first[r] <= j, for j < first[n]: the request that entry j belongs to
// (requests without entries share their start with the next one and are passed over).
__device__ __forceinline__ int owner(const int32_t *first, int n, int32_t j) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= j) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) kv_layout_kernel(const __grid_constant__ mlora_kv_batch b, FastDiv pt,
                                                             int32_t *status) {
  extern __shared__ __align__(16) char smem[];
  LayoutSmem &sh = *reinterpret_cast<LayoutSmem *>(smem);
  const int R = b.num_requests;
  int32_t *rows = reinterpret_cast<int32_t *>(smem + sizeof(LayoutSmem));
  int32_t *pages = rows + R + 1, *back = pages + R + 1, *len = back + R + 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nwarp = blockDim.x >> 5;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t head = b.free_state[0], count = b.free_state[1];
  int bad = 0;
  // thread t holds requests t*each .. t*each+each-1
  const int each = (R + blockDim.x - 1) / blockDim.x;
  int64_t sum[3] = {0, 0, 0};
  const int64_t most = (int64_t)b.max_pages * b.page_tokens;
  for (int k = 0; k < each; ++k) {
    const int r = tid * each + k;
    if (r >= R) break;
    const int32_t l = b.kv_len[r], n = b.new_tokens[r];
    int32_t nr = 0, np = 0, nb = 0;
    if (l < 0 || n < -1 || (int64_t)l + max(n, 0) > most) {
      bad = MLORA_STATUS_BAD_LENGTH;
    } else if (n >= 0) {
      nr = n;
      np = ceil_by(pt, l + n) - ceil_by(pt, l);
    } else {
      nb = ceil_by(pt, l);
    }
    len[r] = l;
    rows[r] = nr;
    pages[r] = np;
    back[r] = nb;
    sum[0] += nr;
    sum[1] += np;
    sum[2] += nb;
  }
  // exclusive sums over the threads: within the warp, then over the warps
  int64_t incl[3] = {sum[0], sum[1], sum[2]};
#pragma unroll
  for (int d = 1; d < 32; d <<= 1)
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      const int64_t o = __shfl_up_sync(~0u, incl[q], d);
      if (lane >= d) incl[q] += o;
    }
  if (lane == 31)
    for (int q = 0; q < 3; ++q) sh.warp[q][warp] = incl[q];
  bad = __syncthreads_or(bad) ? MLORA_STATUS_BAD_LENGTH : 0;  // only that kind so far
  if (warp == 0) {
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      const int64_t own = lane < nwarp ? sh.warp[q][lane] : 0;
      int64_t v = own;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(~0u, v, d);
        if (lane >= d) v += o;
      }
      if (lane < nwarp) sh.warp[q][lane] = v - own;
      if (lane == 31) sh.total[q] = v;
    }
  }
  __syncthreads();
  const int64_t nrow = sh.total[0], npop = sh.total[1], npush = sh.total[2];
  if (nrow > b.num_rows || head < 0 || head >= b.num_pages || count < 0 || count > b.num_pages)
    bad |= MLORA_STATUS_BAD_LENGTH;
  if (!bad && npop > count) bad |= MLORA_STATUS_NO_PAGES;
  if (!bad && count + npush > b.num_pages) bad |= MLORA_STATUS_BAD_LENGTH;
  if (!bad) {
    int64_t at[3];
#pragma unroll
    for (int q = 0; q < 3; ++q) at[q] = sh.warp[q][warp] + incl[q] - sum[q];
    for (int k = 0; k < each; ++k) {  // each thread turns its own requests' counts into starts
      const int r = tid * each + k;
      if (r >= R) break;
      const int32_t nr = rows[r], np = pages[r], nb = back[r];
      rows[r] = (int32_t)at[0];
      pages[r] = (int32_t)at[1];
      back[r] = (int32_t)at[2];
      at[0] += nr;
      at[1] += np;
      at[2] += nb;
    }
    if (tid == 0) {
      rows[R] = (int32_t)nrow;
      pages[R] = (int32_t)npop;
      back[R] = (int32_t)npush;
    }
  }
  __syncthreads();

  const int g = blockIdx.x * blockDim.x + tid, step = gridDim.x * blockDim.x;
  const int32_t P = b.num_pages;
  const int64_t used = bad ? 0 : nrow;
  int report_bits = bad;
  if (!bad) {
    for (int j = g; j < npop; j += step) {  // new page table entries
      const int r = owner(pages, R, j);
      const int32_t first = ceil_by(pt, len[r]);
      int64_t e = head + j;
      if (e >= P) e -= P;
      b.page_table[(int64_t)r * b.table_stride + first + (j - pages[r])] = b.free_ring[e];
    }
    for (int j = g; j < npush; j += step) {  // pages given back
      const int r = owner(back, R, j);
      int64_t e = head + count + j;
      while (e >= P) e -= P;
      b.free_ring[e] = b.page_table[(int64_t)r * b.table_stride + (j - back[r])];
    }
  }
  for (int64_t i = g; i < b.num_rows; i += step) {
    int32_t req = -1, pos = -1, slot = -1;
    int64_t cell = -1;
    if (i < used) {
      req = owner(rows, R, (int32_t)i);
      pos = len[req] + ((int32_t)i - rows[req]);
      const int32_t page = div_by(pt, pos), have = ceil_by(pt, len[req]);
      int32_t id;
      if (page < have) {
        id = b.page_table[(int64_t)req * b.table_stride + page];
      } else {  // a page this call takes: from the ring, as its table entry may not be written yet
        int64_t e = head + pages[req] + (page - have);
        if (e >= P) e -= P;
        id = b.free_ring[e];
      }
      if (id >= 0 && id < P) cell = (int64_t)id * pt.d + (pos - page * pt.d);
      else report_bits |= MLORA_STATUS_BAD_PAGE;
      if (b.adapter_slot) slot = b.adapter_slot[req];
    }
    b.row_request[i] = req;
    b.position[i] = pos;
    b.cache_slot[i] = cell;
    if (b.row_slot) b.row_slot[i] = slot;
  }
  for (int r = g; r <= R; r += step) {
    if (b.seg_offsets) b.seg_offsets[r] = bad ? 0 : rows[r];
    if (b.seg_slot) b.seg_slot[r] = (r < R && b.adapter_slot) ? b.adapter_slot[r] : -1;
  }
  if (g == 0 && b.seg_offsets) b.seg_offsets[R + 1] = b.num_rows;
  if (report_bits) report(status, report_bits);
  // every CTA has read kv_len and free_state
  if (gridDim.x > 1) cluster_sync();
  for (int r = g; r < R; r += step) {
    const int32_t l = len[r];
    // rows[r + 1] - rows[r] = n for n >= 0; a leaving request is the only one with n < 0
    b.kv_len_out[r] = bad ? l : b.new_tokens[r] < 0 ? 0 : l + (rows[r + 1] - rows[r]);
  }
  if (g == 0) {
    b.free_state_out[0] = (int32_t)(bad ? head : (head + npop) % P);
    b.free_state_out[1] = (int32_t)(bad ? count : count - npop + npush);
  }
}

}  // namespace

cudaError_t launch_kv_layout(const mlora_kv_batch &b, int32_t *status, cudaStream_t stream) {
  const size_t smem = sizeof(LayoutSmem) + (size_t)(4 * b.num_requests + 3) * sizeof(int32_t);
  static_assert(sizeof(LayoutSmem) + (4 * MLORA_KV_MAX_REQUESTS + 3) * 4 <= 227 * 1024, "the sums fit in shared memory");
  cudaError_t e = raise_smem<kv_layout_kernel>(227 * 1024);
  if (e != cudaSuccess) return e;
  const int cluster = 8;
  e = launch_waiting(kv_layout_kernel, dim3(cluster), dim3(kThreads), smem, cluster, stream, b, fast_div(b.page_tokens),
                     status);
  if (e == cudaSuccess) api_count_launch();
  return e;
}

}  // namespace mlora
