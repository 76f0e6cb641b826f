// sample.cu -- the next token of each row from a given random number, with temperature, top-k, top-p and min-p (sm_103a).
//
// Every limit, and the token itself, is a place in the row's order (logits descending, then ids): the k-th, or the first at
// which the weights' running sum reaches a number. A place is found without sorting the row: a histogram of counts and weights
// over the logarithm of the weight says in which bin it lies, and only that bin's tokens (with those before it where they are
// few: they serve the next limits, too) are gathered, sorted and summed. Weights and sums are whole numbers
// (sample_weight.cuh), so that the atomics' order does not matter.
//
// A cluster of 1 to 8 CTAs takes a row, each a stretch of its vocabulary: held as fp32 in shared memory where that fits, else
// streamed through a ring of cp.async for each pass (two CTAs an SM, so that one row's chain hides another's). The first CTA does
// the searching; the others count, reduce and gather for it: it writes a command into its shared memory, and all meet at the
// cluster's barrier before and behind its execution.
//
// The bins cover kRangeOfK log2 units with top_k and kRangeOfSum where the sum of all weights is asked for; smaller weights are
// one last bin, summed in registers. Tokens within kNear units of the largest are listed as they are counted: in
// most rows that list answers everything. With top_k the weights are worked out up to the bin of the k-th token only. A bin of
// more than kList tokens, one of many near or equal logits, is divided again by the logits' bits, as often as it
// takes; equal logits are counted by their ids.
//
// One row of 32000: 13.5 us, the chain of loads, meetings and a sort; 21 where the token lies behind the list and a bin has to be gathered.
// 256 rows of 128001 fp32 logits: 266 us (131 MB would be 19 us of memory), bound by the weights of rows that need every token's, shared-memory atomics and the chain of each
// row. Measured there: 1, 2, 4, 8 CTAs a row 436, 290, 267, 290 us; sums kept as three 32-bit parts instead of 64-bit atomics 450
// against 434 us. The two 16-bit variants spill 52 bytes a thread under two CTAs' 64 registers.
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include <algorithm>

#include "sample_weight.cuh"
#include "tc.cuh"

namespace mlora {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 512;           // and one more for what is smaller
// log2 units of the weights that they cover: with top_k, which may ask for tokens of any weight; with the sum of all weights; and
// those whose tokens the CTAs keep as they count them
constexpr float kRangeOfK = 46.f, kRangeOfSum = 24.f, kNear = 8.f;
constexpr int kList = kThreads;     // a thread a token
constexpr int kMaxCtas = 8;
constexpr int kRing = 8;
constexpr int kIdBits = 19;
static_assert(MLORA_SAMPLE_MAX_VOCAB <= 1 << kIdBits, "ids fit the order's code");
static_assert(kBins == kThreads, "a thread a bin");

enum Op { DONE, MASSES, GATHER, DIVIDE, TIES, TIE };
struct Command {
  int32_t op;
  float cut;          // the tokens of a logit of at least cut,
  int32_t lo, hi;     // of the bins lo .. hi,
  uint32_t low, high; // of the keys low .. high
  int32_t shift;      // DIVIDE: keys of a bin, as a power of two, from high down
  int32_t cta, nth;   // TIE
};
constexpr int kCommandWords = sizeof(Command) / 4;

struct Bins {  // counts and weights, or their running sums
  uint32_t count[kBins + 1];
  uint64_t mass[kBins + 1];
};

struct Smem {
  Command cmd;           // written by the first CTA
  float top[kMaxCtas];
  float least;           // min_p as a logit
  uint32_t ties;         // count of TIES
  int32_t found;         // TIE's token; the first token of the largest logit
  int32_t listed;        // tokens of the list; of this CTA's own before
  uint64_t part[kWarps];
  uint32_t cpart[kWarps];
  float2 steps[kExp2Steps];
  Bins bins;             // this CTA's; the first CTA's become the row's
  Bins first, deep;      // the row's running sums: of the first division, of the last of a bin
  uint64_t code[kList], cum[kList];
};

// Key: larger for larger logits. A place in the order is ~key, then the id.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t key) { return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key); }
__device__ __forceinline__ uint64_t code_of(float x, int t) { return (uint64_t)~key_of(x) << kIdBits | (uint32_t)t; }

// The bin of a logit: it does not fall as the logit falls. The last bin's tokens may have weight 0.
__device__ __forceinline__ int bin_of(float x, float top, float scale) {
  const float y = (top - x) * scale;  // (NaN for infinities of one sign)
  return x == top ? 0 : y < (float)kBins ? (int)y : kBins;
}
// No logit below is in a bin up to b: by more than the roundings of bin_of.
__device__ __forceinline__ float cut_of(int b, float top, float scale) {
  if (b >= kBins) return -CUDART_INF_F;
  const float by = (float)(b + 1) / scale;
  return top - by - (by + fabsf(top)) * 0x1p-18f;  // (NaN, where nothing is cut, for an infinite top)
}

__device__ __forceinline__ uint32_t dsmem_ld_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint64_t dsmem_ld_u64(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void dsmem_st_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void dsmem_st_u64(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t dsmem_add(uint32_t addr, uint32_t v) {
  uint32_t old;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(addr), "r"(v) : "memory");
  return old;
}

template <int DT>
struct Vec {  // 16 bytes of logits
  static constexpr int N = 8;
  using T = uint16_t;
  static __device__ __forceinline__ void unpack(const uint4 &u, float (&f)[N]) { unpack8<DT>(u, f); }
  static __device__ __forceinline__ float get(T w) { return Elem<DT>::lo(w); }
};
template <>
struct Vec<MLORA_FP32> {
  static constexpr int N = 4;
  using T = float;
  static __device__ __forceinline__ void unpack(const uint4 &u, float (&f)[N]) {
    f[0] = __uint_as_float(u.x), f[1] = __uint_as_float(u.y), f[2] = __uint_as_float(u.z), f[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ float get(T w) { return w; }
};

__device__ __forceinline__ float cleaned(float x) { return x == x ? x + 0.f : -CUDART_INF_F; }  // NaN as -inf, -0 as 0

// What a CTA of the cluster knows of its row.
template <int DT>
struct Row {
  using V = Vec<DT>;
  using T = typename V::T;
  Smem &sh;
  const T *src;     // this CTA's logits
  const float *x;   // and in shared memory, where they are held
  uint4 *ring;      // where not: what is on its way
  int t0, n;        // its first token, how many
  int cta, ctas;
  float top;
  WeightScale scale;
  float bin_scale;

  __device__ __forceinline__ void meet() const {
    if (ctas > 1) cluster_sync();
    else __syncthreads();
  }
  __device__ __forceinline__ uint32_t of(const void *p, int c) const { return dsmem_addr(p, c); }
  __device__ __forceinline__ float at(int i) const { return x ? x[i] : cleaned(V::get(src[i])); }

  // f(four logits, the first one's place in this CTA's) for all of them, in no order; a place before the first or behind the
  // last has -inf. Whole warps. Where the logits are not held, each thread has kRing vectors of 16 bytes on their way into places of
  // its own in shared memory.
  template <class F>
  __device__ __forceinline__ void each4(F f) const {
    const int skew = (int)((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(T));
    if (x) {
      const float4 *from = reinterpret_cast<const float4 *>(x - skew);
      const int vectors = (n + skew + 3) / 4;
#pragma unroll 1
      for (int v0 = 0; v0 < vectors; v0 += kThreads) {
        const int v = v0 + threadIdx.x;
        const float4 u = v < vectors ? from[v] : make_float4(-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F);
        const float w[4] = {u.x, u.y, u.z, u.w};
        f(w, v * 4 - skew);
      }
      return;
    }
    const T *from = src - skew;  // aligned
    auto fetch = [&](int v, int slot) {
      if (v * V::N >= skew && (v + 1) * V::N <= n + skew) tc::cp_async16(&ring[slot * kThreads + threadIdx.x], from + v * V::N, 16);
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll 1
    for (int j = 0; j < kRing; ++j) fetch(threadIdx.x + j * kThreads, j);
    int slot = 0;
#pragma unroll 1
    for (int v0 = 0; v0 * V::N < n + skew; v0 += kThreads) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
      const int v = v0 + threadIdx.x, t = v * V::N - skew;
      float w[V::N];
      if (t >= 0 && t + V::N <= n) {
        V::unpack(ring[slot * kThreads + threadIdx.x], w);
      } else {
#pragma unroll
        for (int e = 0; e < V::N; ++e) w[e] = t + e >= 0 && t + e < n ? V::get(src[t + e]) : -CUDART_INF_F;
      }
      fetch(v + kRing * kThreads, slot);
      slot = (slot + 1) % kRing;
#pragma unroll
      for (int e = 0; e < V::N; e += 4) {
        const float u[4] = {cleaned(w[e]), cleaned(w[e + 1]), cleaned(w[e + 2]), cleaned(w[e + 3])};
        f(u, t + e);
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
  // The same, one by one.
  template <class F>
  __device__ __forceinline__ void each(F f) const {
    each4([&](const float (&v)[4], int i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) f(v[e], i + e);
    });
  }

  __device__ __forceinline__ bool in(const Command &c, float v) const {
    if (v < c.cut) return false;
    const int b = bin_of(v, top, bin_scale);
    return b >= c.lo && b <= c.hi && key_of(v) - c.low <= c.high - c.low;
  }
  __device__ __forceinline__ void weights(const float (&v)[4], uint64_t (&w)[4]) const { weights_of(v, top, scale, sh.steps, w); }
  // (whole warps)
  __device__ __forceinline__ uint64_t weight(float v) const {
    const float x1[1] = {v};
    uint64_t w[1];
    weights_of(x1, top, scale, sh.steps, w);
    return w[0];
  }
  __device__ __forceinline__ void add_mass(int b, uint64_t w) const {
    atomicAdd(reinterpret_cast<unsigned long long *>(&sh.bins.mass[b]), (unsigned long long)w);
  }

  // The running sums of the cluster's counts (and weights) over the bins, in the first CTA.
  template <bool COUNTS, bool MASSES>
  __device__ void sum_bins(Bins &sums) {
    meet();
    if (cta != 0) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto row_of = [&](int b, uint32_t &count, uint64_t &mass) {
      uint32_t k[kMaxCtas];
      uint64_t m[kMaxCtas];
#pragma unroll
      for (int c = 0; c < kMaxCtas; ++c) {  // all on their way before the first is added
        if (COUNTS) k[c] = c < ctas ? dsmem_ld_u32(of(&sh.bins.count[b], c)) : 0;
        if (MASSES) m[c] = c < ctas ? dsmem_ld_u64(of(&sh.bins.mass[b], c)) : 0;
      }
      count = 0, mass = 0;
#pragma unroll
      for (int c = 0; c < kMaxCtas; ++c) {
        if (COUNTS) count += k[c];
        if (MASSES) mass += m[c];
      }
    };
    uint32_t count, last_count = 0;
    uint64_t mass, last_mass = 0;
    row_of(tid, count, mass);
    if (tid == kThreads - 1) row_of(kBins, last_count, last_mass);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t c = COUNTS ? __shfl_up_sync(~0u, count, d) : 0;
      const uint64_t m = MASSES ? __shfl_up_sync(~0u, mass, d) : 0;
      if (lane >= d) count += c, mass += m;
    }
    if (lane == 31) sh.cpart[warp] = count, sh.part[warp] = mass;
    __syncthreads();
    for (int w = 0; w < warp; ++w) count += sh.cpart[w], mass += sh.part[w];
    if (COUNTS) sums.count[tid] = count;
    if (MASSES) sums.mass[tid] = mass;
    if (tid == kThreads - 1) {
      if (COUNTS) sums.count[kBins] = count + last_count;
      if (MASSES) sums.mass[kBins] = mass + last_mass;
    }
    __syncthreads();
  }

  // Adds to the last bin's weight what the threads hold of it.
  __device__ __forceinline__ void add_last(uint64_t mass) {
#pragma unroll
    for (int d = 16; d; d >>= 1) mass += __shfl_xor_sync(~0u, mass, d);
    if ((threadIdx.x & 31) == 0 && mass) add_mass(kBins, mass);
  }

  // Every CTA of the cluster executes the first one's command.
  __device__ void execute(const Command &c) {
    const int tid = threadIdx.x;
    if (c.op == MASSES) {  // the weights of the first division's bins 0 .. hi
      for (int i = tid; i <= kBins; i += kThreads) sh.bins.mass[i] = 0;
      __syncthreads();
      uint64_t last = 0;
      each4([&](const float (&v)[4], int) {
        bool any = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) any |= !(v[e] < c.cut);
        if (!__any_sync(~0u, any)) return;
        uint64_t w[4];
        weights(v, w);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int b = bin_of(v[e], top, bin_scale);
          if (b > c.hi) continue;
          if (b == kBins) last += w[e];
          else add_mass(b, w[e]);
        }
      });
      add_last(last);
      sum_bins<false, true>(sh.first);
    } else if (c.op == GATHER) {
      const uint32_t counter = of(&sh.listed, 0);
      each([&](float v, int i) {
        if (!in(c, v) || (uint32_t)i >= (uint32_t)n) return;
        const uint32_t at = dsmem_add(counter, 1);
        if (at < (uint32_t)kList) dsmem_st_u64(of(&sh.code[at], 0), code_of(v, t0 + i));
      });
    } else if (c.op == DIVIDE) {
      for (int i = tid; i <= kBins; i += kThreads) sh.bins.count[i] = 0, sh.bins.mass[i] = 0;
      __syncthreads();
      each4([&](const float (&v)[4], int) {
        bool any = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) any |= !(v[e] < c.cut);
        if (!__any_sync(~0u, any)) return;
        uint64_t w[4];
        weights(v, w);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (!in(c, v[e])) continue;
          const uint32_t b = (c.high - key_of(v[e])) >> c.shift;
          atomicAdd(&sh.bins.count[b], 1u);
          add_mass(b, w[e]);
        }
      });
      sum_bins<true, true>(sh.deep);
    } else if (c.op == TIES) {
      uint32_t ties = 0;
      each([&](float v, int i) { ties += in(c, v) && (uint32_t)i < (uint32_t)n; });
      if (tid == 0) sh.ties = 0;
      __syncthreads();
      ties = __reduce_add_sync(~0u, ties);
      if ((tid & 31) == 0) atomicAdd(&sh.ties, ties);
    } else if (c.op == TIE && c.cta == cta) {
      // the nth of this CTA's: thread by thread in stretches, so that the order is the ids'
      const int per = (n + kThreads - 1) / kThreads, i0 = min(tid * per, n), i1 = min(i0 + per, n);
      uint32_t ties = 0;
      for (int i = i0; i < i1; ++i) ties += in(c, at(i));
      uint32_t before = ties;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t o = __shfl_up_sync(~0u, before, d);
        if ((tid & 31) >= d) before += o;
      }
      if ((tid & 31) == 31) sh.cpart[tid >> 5] = before;
      __syncthreads();
      before -= ties;
      for (int w = 0; w < tid >> 5; ++w) before += sh.cpart[w];
      if ((uint32_t)c.nth >= before && (uint32_t)c.nth < before + ties)
        for (int i = i0; i < i1; ++i)
          if (in(c, at(i)) && before++ == (uint32_t)c.nth) dsmem_st_u32(of(&sh.found, 0), (uint32_t)(t0 + i));
    }
  }

  // ---- the first CTA ------------------------------------------------------------------------------------
  __device__ void send(const Command &c) {
    if (threadIdx.x < (unsigned)ctas) {
      const uint32_t to = of(&sh.cmd, threadIdx.x);
#pragma unroll
      for (int i = 0; i < kCommandWords; ++i) dsmem_st_u32(to + i * 4, reinterpret_cast<const uint32_t *>(&c)[i]);
    }
    meet();
  }
  __device__ void command(const Command &c) {
    send(c);
    execute(c);
    meet();
  }

  // Gathers, sorts and sums tokens of which there are at most kList, with `mass` before them.
  __device__ void list(const Command &c, uint64_t mass) {
    if (threadIdx.x == 0) sh.listed = 0;
    command(c);
    sort(min(sh.listed, kList), mass);
  }
  __device__ void sort(int m, uint64_t mass) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int size = 32;
    while (size < m) size <<= 1;
    // bitonic, a token a thread: between the lanes of a warp, and through shared memory where they are further apart
    uint64_t own = tid < m ? sh.code[tid] : ~0ull;
    for (int run = 2; run <= size; run <<= 1)
      for (int step = run >> 1; step; step >>= 1) {
        uint64_t other;
        if (step < 32) {
          other = __shfl_xor_sync(~0u, own, step);
        } else {
          __syncthreads();
          sh.code[tid] = own;
          __syncthreads();
          other = sh.code[tid ^ step];
        }
        const bool smaller = ((tid & step) == 0) == ((tid & run) == 0);
        if ((other < own) == smaller) own = other;
      }
    __syncthreads();
    uint64_t w = weight(tid < m ? logit_of(~(uint32_t)(own >> kIdBits)) : top);
    if (tid >= m) w = 0;
    uint64_t incl = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint64_t o = __shfl_up_sync(~0u, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) sh.part[warp] = incl;
    __syncthreads();
    mass += incl;
    for (int v = 0; v < warp; ++v) mass += sh.part[v];
    sh.code[tid] = own, sh.cum[tid] = mass;
    __syncthreads();
  }

  // How many of the first `m` pass: all of them pass up to a place and none behind it.
  template <class F>
  __device__ int first_that_fails(int m, F passes) const {
    return __syncthreads_count((int)threadIdx.x < m && passes((int)threadIdx.x));
  }

  struct Place {
    uint64_t mass;  // of the order up to and with it
    int token;
  };
  enum Kind { COUNT, MASS, KEY };
  int list_lo = 1, list_hi = 0;  // bins of the first division that the list holds
  int masses_hi = -1;            // up to which bin their weights are there

  __device__ Command bins_of(int op, int lo, int hi) const { return Command{op, cut_of(hi, top, bin_scale), lo, hi, 0, ~0u, 0, 0, 0}; }
  // The first bins up to bin `b`, or as many as fit the list. Those near the largest logit have been kept as they were counted, where
  // they are few.
  __device__ void list_first(int b, bool wanted, int near) {
    if (sh.first.count[near - 1] <= (uint32_t)kList && (b < near || !wanted)) {
      const int tid = threadIdx.x;
      int before = 0, own = 0, from = 0;
      for (int c = 0; c < ctas; ++c) {  // token tid of all
        const int here = (int)dsmem_ld_u32(of(&sh.listed, c));
        if (tid >= before && tid < before + here) own = tid - before, from = c;
        before += here;
      }
      const uint64_t code = tid < before ? dsmem_ld_u64(of(&sh.code[own], from)) : 0;
      __syncthreads();
      sh.code[tid] = code;
      if (tid == 0) sh.listed = before;
      __syncthreads();
      sort(before, 0);
      list_lo = 0, list_hi = near - 1;
      return;
    }
    const int fit = first_that_fails(kBins, [&](int i) { return sh.first.count[i] <= (uint32_t)kList; }) - 1;
    if (fit < 0 || (wanted && fit < b)) return;
    list(bins_of(GATHER, 0, min(b, fit)), 0);
    list_lo = 0, list_hi = min(b, fit);
  }
  // No logit above is in a bin behind b.
  __device__ float bin_end(int b) const {
    const float by = (float)(b + 1) / bin_scale;
    return top - by + (by + fabsf(top)) * 0x1p-18f;
  }
  __device__ int bin_of_count(uint64_t k) const {
    return first_that_fails(kBins, [&](int i) { return sh.first.count[i] < k; });
  }
  // Whether the list from the first token on answers by itself.
  __device__ bool listed(Kind kind, uint64_t arg) const {
    if (list_lo != 0 || list_hi < 0) return false;
    if (kind == COUNT) return sh.first.count[list_hi] >= arg;
    if (kind == KEY) return bin_of(logit_of((uint32_t)arg), top, bin_scale) <= list_hi;
    const int m = min(sh.listed, kList);
    return m > 0 && sh.cum[m - 1] >= arg;
  }

  // COUNT: the place of the arg-th token; MASS: the first at which the running sum reaches arg; KEY: the sum over the logits with
  // a key of at least arg (no token). There is such a place: arg is within the row's sums.
  __device__ Place find(Kind kind, uint64_t arg) {
    if (listed(kind, arg)) return in_list(kind, arg, 0, 0);
    const Bins &s = sh.first;
    int b = kind == KEY ? bin_of(logit_of((uint32_t)arg), top, bin_scale) : kind == COUNT ? bin_of_count(arg) : -1;
    need_masses(b < 0 ? (masses_hi < 0 ? kBins : masses_hi) : b);
    if (b < 0) b = min(first_that_fails(kBins, [&](int i) { return s.mass[i] < arg; }), masses_hi);
    const uint32_t count = b ? s.count[b - 1] : 0;
    const uint64_t mass = b ? s.mass[b - 1] : 0;
    if (b < list_lo || b > list_hi) {
      if (s.count[b] - count > (uint32_t)kList) return find_deep(kind, arg, b, count, mass);
      list(bins_of(GATHER, b, b), mass);
      list_lo = list_hi = b;
    }
    return in_list(kind, arg, list_lo ? s.count[list_lo - 1] : 0, list_lo ? s.mass[list_lo - 1] : 0);
  }
  __device__ void need_masses(int b) {
    if (masses_hi >= b) return;
    command(bins_of(MASSES, 0, b));
    masses_hi = b;
  }

  __device__ Place in_list(Kind kind, uint64_t arg, uint32_t count, uint64_t mass) {
    const int m = min(sh.listed, kList);
    const int p = kind == COUNT ? (int)(arg - 1 - count)
                                : first_that_fails(m, [&](int i) {
                                    return kind == MASS ? sh.cum[i] < arg : ~(uint32_t)(sh.code[i] >> kIdBits) >= (uint32_t)arg;
                                  });
    if (kind == KEY) return Place{p ? sh.cum[p - 1] : mass, -1};
    return Place{sh.cum[p], (int)(sh.code[p] & ((1u << kIdBits) - 1))};
  }

  // The same in a bin of more than kList tokens, with `count` and `mass` before it.
  __device__ Place find_deep(Kind kind, uint64_t arg, int bin, uint32_t count, uint64_t mass) {
    list_lo = 1, list_hi = 0;
    Command c = bins_of(DIVIDE, bin, bin);
    // keys that the bin's lie between
    uint32_t low = key_of(c.cut == c.cut ? c.cut : -CUDART_INF_F), high = key_of(top);
    if (bin > 0) {
      const float before = bin_end(bin - 1);
      if (before < top) high = key_of(before + 0.f);
    }
    for (;;) {
      if (low == high) return find_tie(kind, arg, low, count, mass);
      int shift = 0;
      while ((high - low) >> shift >= (uint32_t)kBins) ++shift;
      c.op = DIVIDE, c.low = low, c.high = high, c.shift = shift;
      command(c);
      const Bins &s = sh.deep;
      const int b = kind == KEY ? (uint32_t)arg > high ? 0 : (int)((high - max((uint32_t)arg, low)) >> shift)
                                : first_that_fails(kBins - 1, [&](int i) { return kind == COUNT ? count + s.count[i] < arg : mass + s.mass[i] < arg; });
      const uint32_t inside = s.count[b] - (b ? s.count[b - 1] : 0);
      if (b) count += s.count[b - 1], mass += s.mass[b - 1];
      const uint32_t top_key = high - ((uint32_t)b << shift);
      low = max(low, top_key - ((1u << shift) - 1u)), high = top_key;
      if (inside <= (uint32_t)kList) {
        __syncthreads();
        c.op = GATHER, c.low = low, c.high = high, c.cut = logit_of(low);
        list(c, mass);
        return in_list(kind, arg, count, mass);
      }
      __syncthreads();
    }
  }

  // The same among more than kList equal logits: the first of their ids.
  __device__ Place find_tie(Kind kind, uint64_t arg, uint32_t key, uint32_t count, uint64_t mass) {
    const uint64_t w = weight(logit_of(key));
    Command c{TIES, logit_of(key), 0, kBins, key, key, 0, 0, 0};
    command(c);
    uint32_t ties = 0;
    for (int i = 0; i < ctas; ++i) ties += dsmem_ld_u32(of(&sh.ties, i));
    if (kind == KEY) return Place{mass + ((uint32_t)arg <= key ? ties * w : 0), -1};
    // (w is not 0 where a sum is reached among them)
    uint64_t nth = kind == COUNT ? arg - 1 - count : w ? (arg - mass - 1) / w : 0;
    const uint64_t up_to = mass + (nth + 1) * w;
    int at = 0;
    for (; at < ctas - 1; ++at) {
      const uint32_t here = dsmem_ld_u32(of(&sh.ties, at));
      if (nth < here) break;
      nth -= here;
    }
    c.op = TIE, c.cta = at, c.nth = (int)nth;
    __syncthreads();
    command(c);
    return Place{up_to, sh.found};
  }
};

template <int DT>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ mlora_sampling p, int32_t row0, int32_t ctas,
                                                             int32_t stretch, bool hold, int32_t *status) {
  using V = Vec<DT>;
  using T = typename V::T;
  extern __shared__ __align__(16) uint8_t raw[];
  Smem &sh = *reinterpret_cast<Smem *>(raw);
  float *held = reinterpret_cast<float *>(raw + (sizeof(Smem) + 15) / 16 * 16);
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = row0 + blockIdx.x / ctas;
  const int cta = blockIdx.x % ctas;
  const int r = p.row_request ? p.row_request[row] : (int)row;
  if (r < 0 || r >= p.num_requests) {  // (all CTAs of the cluster)
    if (r != -1 && cta == 0 && tid == 0) report(status, MLORA_STATUS_BAD_REQUEST);
    return;
  }
  if (ctas > 1) cluster_arrive_relaxed();  // waited for before the first access to another CTA's shared memory
  // ---- the largest logit; the stretch into shared memory, as fp32, where 16-byte vectors of it are aligned ----------
  const int t0 = cta * stretch, n = max(0, min(stretch, p.vocab - t0));
  const T *src = static_cast<const T *>(p.logits) + row * p.ld + t0;
  const int skew = (int)((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(T));
  Row<DT> me{sh, src, nullptr, reinterpret_cast<uint4 *>(held), t0, n, cta, ctas};
  float top = -CUDART_INF_F;
  if (hold) {
    float *x = held + skew;
#pragma unroll 4
    for (int v = tid; v * V::N < n + skew; v += kThreads) {
      const int t = v * V::N - skew;
      float f[V::N];
      if (t >= 0 && t + V::N <= n) {
        V::unpack(ldg_u4(src + t), f);
      } else {
#pragma unroll
        for (int e = 0; e < V::N; ++e) f[e] = t + e >= 0 && t + e < n ? V::get(src[t + e]) : -CUDART_INF_F;
      }
#pragma unroll
      for (int e = 0; e < V::N; ++e) f[e] = cleaned(f[e]), top = fmaxf(top, f[e]);
#pragma unroll
      for (int e = 0; e < V::N; e += 4) *reinterpret_cast<float4 *>(x + t + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
    }
    me.x = x;
  } else {
    me.each([&](float v, int) { top = fmaxf(top, v); });
  }
  float temp = p.temperature ? p.temperature[r] : 1.f;
  int k = p.top_k ? p.top_k[r] : 0;
  if (temp > 0.f) temp = fmaxf(temp, 0x1p-126f);
  else temp = 1.f, k = 1;
  const float limit = p.top_p ? p.top_p[r] : 1.f, least_p = p.min_p ? p.min_p[r] : 0.f;
  for (int i = tid; i < kExp2Steps; i += kThreads) sh.steps[i] = exp2_steps[i];
  for (int i = tid; i <= kBins; i += kThreads) sh.bins.count[i] = 0, sh.bins.mass[i] = 0;
#pragma unroll
  for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
  if (lane == 0) sh.cpart[warp] = __float_as_uint(top);
  __syncthreads();
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, __uint_as_float(sh.cpart[w]));
  if (ctas > 1) {
    cluster_wait();
    if (tid < ctas) dsmem_st_u32(dsmem_addr(&sh.top[cta], tid), __float_as_uint(top));
    cluster_sync();
    for (int c = 0; c < ctas; ++c) top = fmaxf(top, sh.top[c]);
  }
  me.top = top, me.scale = weight_scale(temp);
  const bool sum_all = k <= 0 && (limit < 1.f || !(least_p > 0.f));  // whether the limits begin with the sum of all weights
  const float range = k > 0 ? kRangeOfK : kRangeOfSum;
  const int near = (int)(kBins * kNear / range);
  me.bin_scale = fminf(me.scale.hi * (kBins / range), 3e38f);
  int token = -1;
  float logprob = -CUDART_INF_F;
  if (top != -CUDART_INF_F && k == 1) {
    // ---- the first token of the order ------------------------------------------------------------------------------
    int first = INT32_MAX;
    me.each([&](float v, int i) {
      if (v == top) first = min(first, t0 + i);
    });
    if (tid == 0) sh.found = INT32_MAX;
    __syncthreads();
    first = __reduce_min_sync(~0u, first);
    if (lane == 0 && first != INT32_MAX) atomicMin(&sh.found, first);
    me.meet();
    token = INT32_MAX, logprob = 0.f;
    if (cta == 0)
      for (int c = 0; c < ctas; ++c) token = min(token, (int)dsmem_ld_u32(dsmem_addr(&sh.found, c)));
    if (ctas > 1) cluster_sync();
  } else if (top != -CUDART_INF_F) {
    // ---- counts by bins; the sum of all weights, where it is asked for -----------------------------------------------------
    const bool has_k = k > 0, has_p = limit < 1.f, has_min = least_p > 0.f;
    if (cta == 0 && tid == kThreads - 1 && has_min && least_p < 1.f)
      sh.least = __double2float_ru((double)top + (double)temp * log((double)least_p));
    {
      const float cut = cut_of(kBins - 1, top, me.bin_scale);
      if (tid == 0) sh.listed = 0;
      __syncthreads();
      uint64_t last = 0;
      me.each4([&](const float (&v)[4], int i) {
        uint64_t w[4];
        if (sum_all) me.weights(v, w);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int b = v[e] < cut ? kBins : bin_of(v[e], top, me.bin_scale);
          if (b < kBins) {
            atomicAdd(&sh.bins.count[b], 1u);
            if (sum_all) me.add_mass(b, w[e]);
            if (b < near && *reinterpret_cast<volatile int32_t *>(&sh.listed) < kList) {
              const int at = atomicAdd(&sh.listed, 1);
              if (at < kList) sh.code[at] = code_of(v[e], t0 + i + e);
            }
          } else if (sum_all) {
            last += w[e];
          }
        }
      });
      if (sum_all) me.add_last(last);
      if (sum_all) me.template sum_bins<true, true>(sh.first);
      else me.template sum_bins<true, false>(sh.first);
      me.masses_hi = sum_all ? kBins : -1;
      if (cta == 0 && tid == 0) sh.first.count[kBins] = (uint32_t)p.vocab;  // (the last bin is not counted)
      if (cta == 0) __syncthreads();
    }
    if (cta == 0) {
      // ---- the limits, each a shorter prefix of the order, and the token ------------------------------------
      const float least = least_p < 1.f ? sh.least : top;
      const int least_bin = has_min && least_p <= 1.f ? bin_of(least, top, me.bin_scale) : kBins;
      const bool all_k = !has_k || k >= p.vocab;
      const int k_bin = all_k ? kBins : me.bin_of_count((uint64_t)k);
      if (!all_k) me.list_first(k_bin, true, near);
      else if (has_min && !has_p) me.list_first(least_bin, true, near);
      else me.list_first(kBins - 1, false, near);
      uint64_t kept = ~0ull;
      if (sum_all) {
        kept = sh.first.mass[kBins];
      } else if (!all_k) {
        kept = me.find(Row<DT>::COUNT, (uint64_t)k).mass;
      } else if (has_p || least_bin == kBins) {
        me.need_masses(kBins);
        kept = sh.first.mass[kBins];
      }
      if (has_p) {
        const uint64_t goal = times_ceil(fmaxf(limit, 0.f), kept);
        kept = me.find(Row<DT>::MASS, goal > 0 ? goal : 1).mass;
      }
      if (has_min) {
        uint64_t above = kWeightOne;  // at least the first token
        if (least_p <= 1.f && least_bin > k_bin) above = kept;
        else if (least_p <= 1.f) above = max(me.find(Row<DT>::KEY, key_of(least + 0.f)).mass, kWeightOne);
        kept = min(kept, above);
      }
      const float u = p.uniform[row];
      const uint64_t goal = times_floor(u > 0.f ? fminf(u, 1.f - 0x1p-24f) : 0.f, kept) + 1;
      token = me.find(Row<DT>::MASS, goal).token;
      if (tid == 0) {
        float y = 0.f, yl = 0.f;
        const float chosen = cleaned(V::get(static_cast<const T *>(p.logits)[row * p.ld + token]));
        if (chosen != top) weight_log2(chosen, top, me.scale, y, yl);
        logprob = (y + yl) * 0.693147182f - log1pf((float)(kept - kWeightOne) * (1.f / (float)kWeightOne));
      }
      if (ctas > 1) me.send(Command{DONE});
    } else {
      for (;;) {
        me.meet();
        const Command c = sh.cmd;
        if (c.op == DONE) break;
        me.execute(c);
        me.meet();
      }
    }
  }
  if (cta == 0 && tid == 0) {
    p.token[row] = token;
    if (p.logprob) p.logprob[row] = logprob;
  }
}

constexpr size_t smem_bytes(int stretch) { return (sizeof(Smem) + 15) / 16 * 16 + (size_t)(stretch + 16) * sizeof(float); }
constexpr int kMaxSmem = 227 * 1024;

template <int DT>
cudaError_t launch(const mlora_sampling &p, int32_t *status, cudaStream_t stream) {
  // Stretches of at most 16384 tokens, unless that makes more than eight CTAs for an SM; more CTAs where the rows leave SMs without two.
  // 256 x 128001 with 1, 2, 4, 8 CTAs a row: 436, 290, 267, 290 us; 256 x 32000 100, 85, 100, 139; 64 x 60000 150, 73, 59, 61; 1 x 32000 23,
  // 19, 15, 13.
  int ctas = 1;
  const int64_t sms = sm_count();
  while (ctas < kMaxCtas && ((p.vocab > 16384 * ctas && (int64_t)p.num_rows * ctas * 2 <= 8 * sms) ||
                             ((int64_t)p.num_rows * ctas * 2 <= 2 * sms && p.vocab >= 2048 * ctas)))
    ctas *= 2;
  const int stretch = ((p.vocab + ctas - 1) / ctas + 7) & ~7;
  // held in shared memory where that does not cost CTAs their SM, read again (from L2, mostly) where it does
  const bool hold = smem_bytes(stretch) <= (((int64_t)p.num_rows * ctas > sms) ? kMaxSmem / 2 - 1024 : kMaxSmem);
  const size_t smem = hold ? smem_bytes(stretch) : smem_bytes(0) + kRing * kThreads * 16;
  cudaError_t e = raise_smem<sample_kernel<DT>>(kMaxSmem);
  if (e != cudaSuccess) return e;
  const int64_t most = INT32_MAX / kMaxCtas;  // CTAs are counted in 31 bits
  for (int64_t row0 = 0; row0 < p.num_rows; row0 += most) {
    const dim3 grid((unsigned)(std::min<int64_t>(most, p.num_rows - row0) * ctas));
    e = launch_waiting(sample_kernel<DT>, grid, dim3(kThreads), smem, ctas, stream, p, (int32_t)row0, ctas, stretch, hold, status);
    if (e != cudaSuccess) return e;
    api_count_launch();
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_sample(const mlora_sampling &p, int32_t *status, cudaStream_t stream) {
  switch (p.dtype) {
    case MLORA_FP32: return launch<MLORA_FP32>(p, status, stream);
    case MLORA_BF16: return launch<MLORA_BF16>(p, status, stream);
    default: return launch<MLORA_FP16>(p, status, stream);
  }
}

}  // namespace mlora
