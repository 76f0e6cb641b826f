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
// stores, and the code's own way into the SM (nothing runs often, so its instructions are fetched from afar:
// with the loops unrolled four times a step of 67 requests took 8 us instead of 5.5). So every CTA forms the
// same sums in its own shared memory, and one short loop over entries of all three kinds is dealt over all
// CTAs' threads. Ring entries popped and pushed, and page table entries read and written, are different
// ones (popped: free before the call; pushed: behind those), so nothing has to wait for another CTA,
// except that kv_len_out and free_state_out may be the inputs, which every CTA reads: a small step is one
// cluster (or one CTA) with a barrier before they are written, a large one as many CTAs as it has work for and,
// where they are the inputs, a second launch of one CTA that writes them.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "serve.cuh"

namespace mlora {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

struct LayoutSmem {  // before the arrays: first [3][num_requests + 1], then len
  int64_t warp[3][kWarps];
};

enum { kEntries = 1, kState = 2 };  // what a launch writes: pages and rows; lengths, the ring's state, segments

__global__ void __launch_bounds__(kThreads) kv_layout_kernel(const __grid_constant__ mlora_kv_batch b, FastDiv pt,
                                                             int what, bool cluster, int32_t *status) {
  extern __shared__ __align__(16) char smem[];
  LayoutSmem &sh = *reinterpret_cast<LayoutSmem *>(smem);
  const int R = b.num_requests, P = b.num_pages;
  // [0] rows, [1] pages taken, [2] pages returned: of each request, then of those before it
  int32_t *first = reinterpret_cast<int32_t *>(smem + sizeof(LayoutSmem)), *len = first + 3 * (R + 1);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nwarp = blockDim.x >> 5;
  pdl_wait();
  pdl_launch_dependents();
  const int head = b.free_state[0], count = b.free_state[1];
  int bad = 0;
  // thread t holds requests r0 .. r1 - 1
  const int each = (R + blockDim.x - 1) / blockDim.x;
  const int r0 = min(tid * each, R), r1 = min(r0 + each, R);
  int64_t sum[3] = {0, 0, 0};
#pragma unroll 4
  for (int r = r0; r < r1; ++r) {
    const int32_t l = b.kv_len[r], n = b.new_tokens[r];
    const bool ok = l >= 0 && n >= -1 && (int64_t)l + max(n, 0) <= (int64_t)b.max_pages * pt.d;
    bad |= !ok;
    const int have = ok ? ceil_by(pt, l) : 0;
    const int c[3] = {ok && n > 0 ? n : 0, ok && n > 0 ? ceil_by(pt, l + n) - have : 0, n < 0 ? have : 0};
    len[r] = l;
#pragma unroll
    for (int q = 0; q < 3; ++q) first[q * (R + 1) + r] = c[q], sum[q] += c[q];
  }
  // exclusive sums over the threads: within the warp, then over the warps
  int64_t at[3];
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    int64_t x = sum[q];
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(~0u, x, d);
      if (lane >= d) x += o;
    }
    at[q] = x - sum[q];
    if (lane == 31) sh.warp[q][warp] = x;
  }
  bad = __syncthreads_or(bad) ? MLORA_STATUS_BAD_LENGTH : 0;
  int64_t total[3];
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    int64_t x = lane < nwarp ? sh.warp[q][lane] : 0;
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(~0u, x, d);
      if (lane >= d) x += o;
    }
    total[q] = __shfl_sync(~0u, x, 31);
    if (warp) at[q] += __shfl_sync(~0u, x, warp - 1);
  }
  if (total[0] > b.num_rows || head < 0 || head >= P || count < 0 || count > P) bad |= MLORA_STATUS_BAD_LENGTH;
  if (!bad && total[1] > count) bad |= MLORA_STATUS_NO_PAGES;
  if (!bad && count + total[2] > P) bad |= MLORA_STATUS_BAD_LENGTH;
  if (!bad) {
#pragma unroll 1
    for (int r = r0; r < r1; ++r)
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        const int c = first[q * (R + 1) + r];
        first[q * (R + 1) + r] = (int32_t)at[q];
        at[q] += c;
      }
  }
  __syncthreads();

  const int g = blockIdx.x * blockDim.x + tid, step = gridDim.x * blockDim.x;
  const int npop = bad ? 0 : (int)total[1], npush = bad ? 0 : (int)total[2], used = bad ? 0 : (int)total[0];
  int report_bits = bad;
  // entries: pages taken, pages returned, rows
  for (int64_t e = g; (what & kEntries) && e < (int64_t)npop + npush + b.num_rows; e += step) {
    const int kind = e < npop ? 1 : e < npop + npush ? 2 : 0;
    const int j = (int)(e - (kind == 1 ? 0 : kind == 2 ? npop : npop + npush));  // among its kind
    const bool row = kind == 0;
    int r = 0, pos = -1, id = -1, slot = -1;
    int64_t ring = 0, cell = 0;  // places of the entry's page in the ring and the table
    if (!row || j < used) {
      // its request: the last that starts at or before it (those without entries are passed over)
      const int32_t *f = first + kind * (R + 1);
      for (int hi = R; hi - r > 1;) {
        const int mid = (r + hi) >> 1;
        if (f[mid] <= j) r = mid;
        else hi = mid;
      }
      const int in = j - f[r], have = ceil_by(pt, len[r]);
      pos = len[r] + in;
      const int page = row ? div_by(pt, pos) : kind == 1 ? have + in : in;
      // a row's page that this call takes comes from the ring, as its table entry may not be written yet
      const bool fresh = kind == 1 || (row && page >= have);
      ring = (int64_t)head + (kind == 2 ? count + j : first[R + 1 + r] + page - have);
      if (ring >= P) ring -= P;
      if (ring >= P) ring -= P;
      cell = (int64_t)r * b.table_stride + page;
      id = fresh ? b.free_ring[ring] : b.page_table[cell];
      if (row && b.adapter_slot) slot = b.adapter_slot[r];
    } else {
      r = -1;
    }
    if (kind == 1) {
      b.page_table[cell] = id;
    } else if (kind == 2) {
      b.free_ring[ring] = id;
    } else {
      const bool good = id >= 0 && id < P;
      if (r >= 0 && !good) report_bits |= MLORA_STATUS_BAD_PAGE;
      b.row_request[j] = r;
      b.position[j] = pos;
      b.cache_slot[j] = good ? (int64_t)id * pt.d + (pos - div_by(pt, pos) * pt.d) : -1;
      if (b.row_slot) b.row_slot[j] = slot;
    }
  }
  if (report_bits) report(status, report_bits);
  if (!(what & kState)) return;
  if (cluster) cluster_sync();  // every CTA has read kv_len and free_state
  for (int r = g; r < R + 2; r += step) {
    const int start = r >= R ? used : bad ? 0 : first[r], n = r >= R ? 0 : b.new_tokens[r];
    if (b.seg_offsets) b.seg_offsets[r] = r > R ? b.num_rows : start;
    if (b.seg_slot && r <= R) b.seg_slot[r] = (r < R && b.adapter_slot) ? b.adapter_slot[r] : -1;
    if (r < R) b.kv_len_out[r] = bad ? len[r] : n < 0 ? 0 : len[r] + n;
  }
  if (g < 2) {
    int x = g ? count : head;
    if (!bad) x = g ? count - npop + npush : head + npop >= P ? head + npop - P : head + npop;
    b.free_state_out[g] = x;
  }
}

}  // namespace

cudaError_t launch_kv_layout(const mlora_kv_batch &b, int32_t *status, cudaStream_t stream) {
  const size_t smem = sizeof(LayoutSmem) + (size_t)(4 * b.num_requests + 3) * sizeof(int32_t);
  static_assert(sizeof(LayoutSmem) + (4 * MLORA_KV_MAX_REQUESTS + 3) * 4 <= 227 * 1024, "the sums fit in shared memory");
  cudaError_t e = raise_smem<kv_layout_kernel>(227 * 1024);
  if (e != cudaSuccess) return e;
  const FastDiv pt = fast_div(b.page_tokens);
  auto run = [&](int ctas, int threads, int what, int cluster) {
    const cudaError_t err = launch_waiting(kv_layout_kernel, dim3(ctas), dim3(threads), smem, cluster, stream, b, pt, what,
                                           cluster > 1, status);
    if (err == cudaSuccess) api_count_launch();
    return err;
  };
  // Rows and requests, of which most have an entry. Measured: 32 decoding requests 3.3 us with one CTA of 256
  // threads, 3.9 with a cluster of eight; 67 requests and 2770 rows 9.8 and 4.2; 4096 requests and 48
  // thousand rows 20 with the cluster, 9.4 with a CTA per 1024 entries (11 per 512, 17 per 256), and 15.8 in place, where the
  // second launch has to follow.
  const int64_t work = (int64_t)b.num_rows + b.num_requests;
  if (work <= 512) return run(1, 256, kEntries | kState, 1);
  if (work <= 8 * 1024) return run(8, 512, kEntries | kState, 8);
  const int ctas = (int)std::min((int64_t)sm_count(), (work + kThreads - 1) / kThreads);
  if (b.kv_len_out != b.kv_len && b.free_state_out != b.free_state) return run(ctas, kThreads, kEntries | kState, 1);
  e = run(ctas, kThreads, kEntries, 1);
  return e == cudaSuccess ? run(1, kThreads, kState, 1) : e;
}

}  // namespace mlora
