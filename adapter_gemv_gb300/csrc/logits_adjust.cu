// logits_adjust.cu -- each request's penalties, biases, temperature and grammar mask on its logits (sm_103a).
//
// Elementwise over [rows][vocab] once the history is a count per token: 2 x 4 bytes a logit and a
// mask bit against a handful of flops, so bound by memory for a batch and by latency for a row.
//
// A CTA takes a slice of one row's vocabulary and streams it through: temperature and mask, which need no
// table. Few of its tokens are in the request's history or bias list. They are worked out behind the
// stream, a thread a token, from the logits as they came, over what the stream has written there. (Where out is
// logits, the bits below are made before the stream, and it leaves those tokens alone.) So the stream needs
// few registers and waits for nothing but the row's parameters, the tables are small, and four CTAs share an
// SM: while one waits for its history or its counts, the others stream.
// A bit per token says which are in the history or the list.
// The touched tokens are numbered by their place among the bits set (a prefix sum over the words), and have
// their count (occurrences past the prompt, whole-number atomics: the order does not matter; bit 31 for a
// token of the prompt) and bias (the entry's number + 1, then its value, as one 64-bit maximum: of several
// with one id the last wins) in arrays by that number; more than kPlaces of them, of a long history, take
// several turns. Each CTA of a row reads the whole history and list, from L2 after the first: once for the bits and
// once more for every kPlaces tokens that it finds in its slice. That is some 16 KB twice for a history of 4096, but it
// grows with the history times the touched tokens of a slice, and the choice of the slices does not look at it. At 128001
// fp32 logits a row with histories of 1, 4096, 32768, 131072 tokens: one row 3.5, 5.8, 25, 154 us; 64 rows 19, 23, 167,
// 1255; 256 rows 50, 71, 567, 4726 (token ids by a power law).
// Measured at 256 x 128001 fp32 with histories of 512 to 4096 tokens, lists of 300 and half the rows masked: 61 us,
// 4.3 TB/s (43 us, 6.1 TB/s, without history, list and mask), 101 us in place, where the bits come before the stream;
// bf16 53 and 105. What is left is the touched tokens' chain: bits
// 4 us, numbers 1, counts 8, their logits 4. Also tried there: a table entry for every token of the slice,
// its logits held in registers until the counts were there, 88 us; the touched tokens adjusted in the stream, with
// the counts before it, 75 to 82; a CTA's share as one long stretch, 76; a list of the slice's tokens in
// shared memory instead of reading the history twice, 69; more CTAs an SM with fewer registers, 64 to 76.
//
// Rows of an odd vocabulary start at any multiple of the element: a slice is cut where 16-byte
// vectors are aligned in memory, counted from the aligned address before the row's start.
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include <algorithm>

#include "serve.cuh"

namespace mlora {

namespace {

template <int DT>
struct Vec {  // a 16-byte vector of logits
  static constexpr int N = 8;
  using T = uint16_t;
  static __device__ __forceinline__ void unpack(const uint4 &u, float (&f)[N]) { unpack8<DT>(u, f); }
  static __device__ __forceinline__ uint4 pack(const float (&f)[N]) { return pack8<DT>(f); }
  static __device__ __forceinline__ float get(T w) { return Elem<DT>::lo(w); }
  static __device__ __forceinline__ T put(float f) { return Elem<DT>::from_float(f); }
};
template <>
struct Vec<MLORA_FP32> {
  static constexpr int N = 4;
  using T = float;
  static __device__ __forceinline__ void unpack(const uint4 &u, float (&f)[N]) {
    f[0] = __uint_as_float(u.x), f[1] = __uint_as_float(u.y), f[2] = __uint_as_float(u.z), f[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[N]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
  static __device__ __forceinline__ float get(T w) { return w; }
  static __device__ __forceinline__ T put(float f) { return f; }
};

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCtasPerSm = 4;
constexpr int kGroup = 4;    // vectors of a thread that are loaded together
constexpr int kEarlyBias = 2;  // and entries of the list
constexpr int kEarly = 4;    // tokens of the history that a thread loads ahead
constexpr int kPlaces = 512;
constexpr uint32_t kInPrompt = 0x80000000u;

template <int SLICE>
struct LogitsSmem {
  static_assert(SLICE + 8 <= INT32_MAX - MLORA_LOGITS_MAX_VOCAB, "tokens up to a slice's end are counted in 31 bits");
  static constexpr int kWords = SLICE / 32;
  uint32_t grammar[kWords + 1];  // the mask's bits of the slice, from the word of its first token
  uint32_t hit[kWords];          // tokens of the history or the list
  uint32_t before[kWords];       // how many of them in earlier words
  uint32_t count[kPlaces], place[kPlaces];
  unsigned long long bias[kPlaces];
  uint32_t warp_sum[kWarps];
};

template <int DT, int G>  // G groups of vectors a thread; G = 0: one vector
__global__ void __launch_bounds__(kThreads, kCtasPerSm) logits_kernel(const __grid_constant__ mlora_logits p, int32_t row0,
                                                          int32_t *status) {
  using V = Vec<DT>;
  using T = typename V::T;
  constexpr int kVecs = G ? G * kGroup : 1, kLoad = G ? kGroup : 1;
  constexpr int kSlice = kThreads * kVecs * V::N;
  using Smem = LogitsSmem<kSlice>;
  __shared__ Smem sh;
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, slice = blockIdx.x;
  const int64_t row = (int64_t)row0 + blockIdx.y;
  int bad = 0;
  const int r = p.row_request ? p.row_request[row] : (int)row;
  if (r < -1 || r >= p.num_requests) bad |= MLORA_STATUS_BAD_REQUEST;
  const T *src = static_cast<const T *>(p.logits) + row * p.ld;
  T *dst = static_cast<T *>(p.out) + row * p.ldo;
  const int skew = (int)((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(T));  // elements before the row's start
  const bool in_place = dst == src;
  const bool same_skew = (int)((reinterpret_cast<uintptr_t>(dst) & 15) / sizeof(T)) == skew;
  const int first = slice * kSlice - skew;  // token of the slice's first place (below 0 in a skewed first slice)
  if (r == -1 || first >= p.vocab) return;
  const int low = max(first, 0), high = min(first + kSlice, p.vocab);  // the slice's tokens
  const bool interior = low == first && high == first + kSlice;

  // Vector i of a thread: a whole one inside the row as it is; else its elements inside, from the first bits on.
  auto token_of = [&](int i) { return first + (i * kThreads + tid) * V::N; };
  auto load = [&](int i) {
    const int t = token_of(i);
    if (interior || (t >= 0 && t + V::N <= p.vocab)) return ldg_u4(src + t);
    float f[V::N];
#pragma unroll
    for (int e = 0; e < V::N; ++e) f[e] = (t + e >= 0 && t + e < p.vocab) ? V::get(src[t + e]) : 0.f;
    return V::pack(f);
  };
  uint4 x[kLoad];
#pragma unroll
  for (int k = 0; k < kLoad; ++k) x[k] = load(k);

  int total = 0, prompt = 0, bias0 = 0, bias1 = 0, grammar = -1;
  float rep = 1.f, pres = 0.f, freq = 0.f, temp = 1.f;
  const int32_t *text = nullptr;
  int early[kEarly] = {};
  if (!bad) {
    if (p.total_len) {
      total = p.total_len[r], prompt = p.prompt_len[r];
      text = p.tokens + (int64_t)r * p.tokens_stride;
#pragma unroll
      for (int k = 0; k < kEarly; ++k)
        if (k * kThreads + tid < p.tokens_len) early[k] = text[k * kThreads + tid];
      if (total < 0 || total > p.tokens_len || prompt < 0 || prompt > total) bad |= MLORA_STATUS_BAD_LENGTH;
    }
    if (p.bias_offsets) {
      bias0 = p.bias_offsets[r], bias1 = p.bias_offsets[r + 1];
      if (bias0 < 0 || bias1 < bias0 || bias1 > p.num_bias) bad |= MLORA_STATUS_BAD_LENGTH;
    }
    if (p.mask) {
      grammar = p.mask_index[r];
      if (grammar < -1 || grammar >= p.num_masks) bad |= MLORA_STATUS_BAD_SLOT;
    }
    if (p.repetition) rep = p.repetition[r];
    if (p.presence) pres = p.presence[r];
    if (p.frequency) freq = p.frequency[r];
    if (p.temperature) temp = p.temperature[r];
    if (!(temp > 0.f)) temp = 1.f;
  }
  if (bad) {
    if (slice == 0 && tid == 0) report(status, bad);
    return;
  }

  // ---- which tokens of the slice are in the history or the list --------------------------------------
  const int listed = bias1 - bias0;
  int early_bias[kEarlyBias];
  float early_value[kEarlyBias];
#pragma unroll
  for (int k = 0; k < kEarlyBias; ++k) {
    const int i = k * kThreads + tid;
    early_bias[k] = i < listed ? p.bias_token[bias0 + i] : 0;
    early_value[k] = i < listed ? p.bias_value[bias0 + i] : 0.f;
  }
  const bool touched = total > 0 || listed > 0;
  const uint32_t *bits = grammar >= 0 ? p.mask + grammar * p.mask_stride : nullptr;
  const int word0 = first >> 5, last_word = (p.vocab - 1) >> 5;  // (first may be below 0)
  if (bits)
    for (int i = tid; i <= Smem::kWords; i += kThreads) sh.grammar[i] = bits[min(max(word0 + i, 0), last_word)];
  auto inside = [&](int t) { return (uint32_t)(t - low) < (uint32_t)(high - low); };
  auto each_token = [&](auto f) {  // of the history, with its place in it
#pragma unroll
    for (int k = 0; k < kEarly; ++k)
      if (k * kThreads + tid < total) f(k * kThreads + tid, early[k]);
#pragma unroll 4
    for (int i = kEarly * kThreads + tid; i < total; i += kThreads) f(i, text[i]);
  };
  auto each_entry = [&](auto f) {  // of the list, with its value
#pragma unroll
    for (int k = 0; k < kEarlyBias; ++k)
      if (k * kThreads + tid < listed) f(k * kThreads + tid, early_bias[k], early_value[k]);
    for (int i = kEarlyBias * kThreads + tid; i < listed; i += kThreads) f(i, p.bias_token[bias0 + i], p.bias_value[bias0 + i]);
  };
  int kept = 0;  // how many tokens
  // counts and biases of the tokens numbered from .. from + kPlaces - 1
  auto number = [&](int t) {
    const uint32_t at = (uint32_t)(t - first), w = at >> 5;
    return sh.before[w] + __popc(sh.hit[w] & ((1u << (at & 31)) - 1u));
  };
  auto count_from = [&](int from) {
    const uint32_t n = (uint32_t)min(kPlaces, kept - from);
    if (from) {  // (for the first turn they were cleared with the bits)
      for (int j = tid; j < kPlaces; j += kThreads) sh.count[j] = 0, sh.bias[j] = 0;
    }
    __syncthreads();
    each_token([&](int i, int t) {
      if (!inside(t)) return;
      const uint32_t j = number(t) - (uint32_t)from;
      if (j >= n) return;
      sh.place[j] = (uint32_t)(t - first);
      if (i < prompt) atomicOr(&sh.count[j], kInPrompt);
      else atomicAdd(&sh.count[j], 1u);
    });
    each_entry([&](int i, int t, float value) {
      if (!inside(t)) return;
      const uint32_t j = number(t) - (uint32_t)from;
      if (j >= n) return;
      sh.place[j] = (uint32_t)(t - first);
      atomicMax(&sh.bias[j], ((unsigned long long)(i + 1) << 32) | __float_as_uint(value));
    });
    __syncthreads();
  };
  auto adjusted = [&](float f, int j) {  // before the temperature
    const uint32_t c = sh.count[j], made = c & ~kInPrompt;
    if (c) f = f > 0.f ? f / rep : f * rep;
    if (made) f = f - freq * (float)made - pres;
    const unsigned long long b = sh.bias[j];
    return b ? f + __uint_as_float((uint32_t)b) : f;
  };
  auto mark_all = [&]() {
    for (int i = tid; i < Smem::kWords; i += kThreads) sh.hit[i] = 0;
    for (int j = tid; j < kPlaces; j += kThreads) sh.count[j] = 0, sh.bias[j] = 0;
    __syncthreads();
    int wrong = 0;
    auto mark = [&](int t) {
      if (slice == 0 && (uint32_t)t >= (uint32_t)p.vocab) wrong = MLORA_STATUS_BAD_TOKEN;
      if (inside(t)) atomicOr(&sh.hit[(t - first) >> 5], 1u << ((t - first) & 31));
    };
    each_token([&](int, int t) { mark(t); });
    each_entry([&](int, int t, float) { mark(t); });
    if (wrong) report(status, wrong);
  };
  if (touched && in_place) mark_all();
  if ((touched && in_place) || bits) __syncthreads();

  // ---- the stream -------------------------------------------------------------------------------------
#pragma unroll 1
  for (int g = 0; g < (G ? G : 1); ++g) {
    uint4 y[kLoad];
#pragma unroll
    for (int k = 0; k < kLoad; ++k) y[k] = x[k];
    if (g + 1 < G) {
#pragma unroll
      for (int k = 0; k < kLoad; ++k) x[k] = load((g + 1) * kGroup + k);
    }
#pragma unroll
    for (int k = 0; k < kLoad; ++k) {
      const int i = g * kGroup + k, at = (i * kThreads + tid) * V::N, t = first + at;
      float f[V::N];
      V::unpack(y[k], f);
      uint32_t allowed = ~0u;  // of the vector's tokens, from bit 0
      if (bits)
        allowed = __funnelshift_r(sh.grammar[(t >> 5) - word0], sh.grammar[((t + V::N - 1) >> 5) - word0], t & 31);
      const uint32_t later = touched && in_place ? (sh.hit[at / 32] >> (at % 32)) & ((1u << V::N) - 1u) : 0u;
#pragma unroll
      for (int e = 0; e < V::N; ++e) {
        f[e] = f[e] / temp;
        if (!(allowed >> e & 1u)) f[e] = -CUDART_INF_F;
      }
      if (same_skew && !later && (interior || (t >= 0 && t + V::N <= p.vocab))) {
        *reinterpret_cast<uint4 *>(dst + t) = V::pack(f);
      } else {
#pragma unroll
        for (int e = 0; e < V::N; ++e)
          if (!(later >> e & 1u) && t + e >= 0 && t + e < p.vocab) dst[t + e] = V::put(f[e]);
      }
    }
  }
  if (!touched) return;
  if (!in_place) mark_all();
  __syncthreads();  // (also: what the stream has written comes before what follows)

  // ---- the touched tokens ------------------------------------------------------------------------------------
  {
    constexpr int kEach = (Smem::kWords + kThreads - 1) / kThreads;  // words a thread counts
    uint32_t n = 0;
#pragma unroll
    for (int k = 0; k < kEach; ++k)
      if (tid * kEach + k < Smem::kWords) n += __popc(sh.hit[tid * kEach + k]);
    uint32_t incl = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t o = __shfl_up_sync(~0u, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) sh.warp_sum[warp] = incl;
    __syncthreads();
    uint32_t at = incl - n, all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) at += sh.warp_sum[w];
      all += sh.warp_sum[w];
    }
    kept = (int)all;
#pragma unroll
    for (int k = 0; k < kEach; ++k)
      if (tid * kEach + k < Smem::kWords) {
        sh.before[tid * kEach + k] = at;
        at += __popc(sh.hit[tid * kEach + k]);
      }
  }
  for (int from = 0; from < kept; from += kPlaces) {  // (one turn, but for long histories)
    if (from) __syncthreads();
    count_from(from);
    for (int j = tid; j < min(kPlaces, kept - from); j += kThreads) {
      const int t = first + (int)sh.place[j];
      float f = adjusted(V::get(src[t]), j) / temp;
      if (bits && !((sh.grammar[(t >> 5) - word0] >> (t & 31)) & 1u)) f = -CUDART_INF_F;
      dst[t] = V::put(f);
    }
  }
}

template <int DT, int G>
cudaError_t launch(const mlora_logits &a, int32_t *status, cudaStream_t stream) {
  constexpr int kSlice = kThreads * (G ? G * kGroup : 1) * Vec<DT>::N;
  // a row may start up to one vector's elements after an aligned address
  const int64_t slices = ((int64_t)a.vocab + Vec<DT>::N - 1 + kSlice - 1) / kSlice;
  for (int64_t row0 = 0; row0 < a.num_rows; row0 += 65535) {  // (the last step may pass 2^31)
    const dim3 grid((unsigned)slices, (unsigned)std::min<int64_t>(65535, a.num_rows - row0));
    const cudaError_t e = launch_waiting(logits_kernel<DT, G>, grid, dim3(kThreads), 0, 1, stream, a, (int32_t)row0, status);
    if (e != cudaSuccess) return e;
    api_count_launch();
  }
  return cudaSuccess;
}

template <int DT>
cudaError_t dispatch(const mlora_logits &a, int32_t *status, cudaStream_t stream) {
  // The longer the slices, the fewer times a row's history is read and counted; the shorter, the more SMs
  // work. All CTAs take about as long, so a last wave of few costs as much as a full one: a call takes
  // ceil(CTAs / resident) times 4 + vectors a thread. Measured (us) with slices of 1, 4, 8 and 16 vectors
  // a thread, fp32 unless said; 16-bit slices have twice the tokens:
  //   4 x 38319: 4.2  5.8  7.5  14.3      24 x 47632: 8.8  6.3  7.5  10.8      64 x 32000: 14.3  7.5  7.9  10.9
  //   32 x 128001: 24.6  12.8  11.9  13.8    64 x 128001: 48.7  23.5  20.4  18.6   256 x 32000: 54.3  24.5  20.3  18.3
  //   256 x 128001: -  -  74.8  61.4    256 x 69248: 140  55.4  46.0  47.2
  //   bf16 8 x 32000: 5.1  6.8  9.7  15.7    fp16 128 x 128001: 56  30  29  27    fp16 213 x 69248: 52  31  36  52
  const int64_t resident = (int64_t)kCtasPerSm * sm_count();
  auto cost = [&](int vectors) {
    const int64_t slice = (int64_t)kThreads * vectors * Vec<DT>::N;
    const int64_t ctas = (int64_t)a.num_rows * (((int64_t)a.vocab + Vec<DT>::N - 1 + slice - 1) / slice);
    return (ctas + resident - 1) / resident * (4 + vectors);
  };
  const int64_t c0 = cost(1), c1 = cost(kGroup), c2 = cost(2 * kGroup), c4 = cost(4 * kGroup);
  const int64_t best = std::min(std::min(c0, c1), std::min(c2, c4));
  if (best == c0) return launch<DT, 0>(a, status, stream);
  if (best == c1) return launch<DT, 1>(a, status, stream);
  if (best == c2) return launch<DT, 2>(a, status, stream);
  return launch<DT, 4>(a, status, stream);
}

}  // namespace

cudaError_t launch_logits_adjust(const mlora_logits &a, int32_t *status, cudaStream_t stream) {
  switch (a.dtype) {
    case MLORA_FP32: return dispatch<MLORA_FP32>(a, status, stream);
    case MLORA_BF16: return dispatch<MLORA_BF16>(a, status, stream);
    default: return dispatch<MLORA_FP16>(a, status, stream);
  }
}

}  // namespace mlora
